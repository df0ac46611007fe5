"""GPU tests of qmv_rope_append_e4m3 on long prompts: from 256 rows on a CTA takes two rows of q, and
there are many windows of k and v. Definition and tolerances as in the operator's own tests."""
import pytest
import torch

from test_gpu_append_e4m3 import check, inputs

pytestmark = pytest.mark.gpu


def prompts(M):
    """M rows: runs that start inside a block and at its start, in pages out of order, rows of padding between and behind."""
    slots, at = [], 3
    while len(slots) < M:
        slots += list(range(at, at + 150)) + [-1] * (len(slots) % 3)
        at = (at // 16 * 16) + 16 * 23 + (at * 7) % 16
        if at + 150 > 16 * 400:
            at = 16 * 9 + 5
    return slots[:M - 1] + [-1] if M % 2 else slots[:M]


@pytest.mark.parametrize("M", [255, 256, 257, 1335])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 1), (64, 40, 2), (128, 5, 1), (128, 17, 2), (128, 32, 1)])
def test_many_rows(D, Hq, Hkv, interleaved, dtype, M):
    slots = prompts(M)
    assert len({s for s in slots if s >= 0}) == sum(s >= 0 for s in slots)     # no slot twice
    args = inputs(slots, D=D, Hq=Hq, Hkv=Hkv, page=64, pages=100, rot=D if Hq % 2 else D // 2, seed=M + Hq, axes=1 + Hq % 3)
    check(args, interleaved=interleaved, dtype=dtype, u=2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8)


def test_three_prompts_of_1335_rows():
    slots = [s for b in range(3) for s in range(1600 * b + 100, 1600 * b + 1435)]
    check(inputs(slots, D=128, Hq=10, Hkv=2, page=64, pages=75, norm=False, seed=5), u=2.0 ** -11)
