"""Appends of codes with the attention over them right behind, no other launch between them: with
programmatic overlap the attention starts while the append writes the codes and scales that it reads."""
import pytest
import torch

from cache8_ref import E4M3

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Hq,Hkv,D,before", [(3, 8, 2, 64, 0), (16, 32, 8, 128, 100), (64, 16, 4, 128, 700)])
def test_steps_without_launches_between_give_the_same_when_they_overlap(B, Hq, Hkv, D, before):
    import gemm_qmv_quantize_gb300 as q
    steps, page = 40, 32
    width = (before + steps + page - 1) // page
    g = torch.Generator(device="cuda").manual_seed(50)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    pages = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).reshape(B, width).contiguous()
    slot = lambda n: (pages[:, n // page].long() * page + n % page).contiguous()  # noqa: E731
    table, w = q.qmv_rope_table(before + steps, D, device="cuda"), r(D)
    prompt, new = r(B * before, (Hq + 2 * Hkv) * D), [r(B, (Hq + 2 * Hkv) * D) * 2.0 ** (n % 5) for n in range(steps)]
    slots = [slot(n) for n in range(before + steps)]
    positions = [torch.full((1, B), n, dtype=torch.int32, device="cuda") for n in range(before + steps)]
    lens = [torch.full((B,), before + n + 1, dtype=torch.int32, device="cuda") for n in range(steps)]
    workspace = torch.empty((q.qmv_paged_attention_e4m3_workspace(B, 1, Hq, Hkv, D, width * page),), dtype=torch.uint8, device="cuda")
    results = []
    for overlap in (False, True):
        k, v = (torch.zeros((B * width, page, Hkv, D), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
        ks, vs = (torch.zeros((B * width, page // 16, Hkv), device="cuda") for _ in range(2))
        qs, outs = ([torch.empty((B, Hq, D), dtype=torch.float16, device="cuda") for _ in range(steps)] for _ in range(2))
        if before:
            q.qmv_rope_append_e4m3(prompt, torch.arange(before, dtype=torch.int32, device="cuda").repeat(1, B), table, bytes(D // 2),
                                   torch.stack(slots[:before], 1).flatten(), k, v, ks, vs, w, w)
        torch.cuda.synchronize()
        try:
            q.set_launch_overlap(overlap)
            for n in range(steps):
                q.qmv_rope_append_e4m3(new[n], positions[before + n], table, bytes(D // 2), slots[before + n], k, v, ks, vs, w, w, out=qs[n])
                q.qmv_paged_attention_e4m3(qs[n].view(B, 1, Hq, D), k, v, ks, vs, pages, lens[n], out=outs[n].view(B, 1, Hq, D),
                                           workspace=workspace)
            torch.cuda.synchronize()
        finally:
            q.set_launch_overlap(False)
        results.append([*qs, *outs, k.view(torch.uint8), v.view(torch.uint8), ks, vs])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert bool(torch.isfinite(results[0][2 * steps - 1]).all())
