"""The smoke pass launches each of the library's operators, those over a cache of 8 bits among them."""
import pytest

pytestmark = pytest.mark.gpu


def test_smoke_runs_every_operator():
    import __graft_entry__
    import gemm_qmv_quantize_gb300 as q
    q.route_reset()
    __graft_entry__.smoke()
    counts = q.route_counts()
    for name in ("lora_add", "rope_append", "prefix_attention", "penalize_logits", "norm_rope_append", "rope_append_e4m3",
                 "paged_attention_e4m3", "sample"):
        assert counts[name] > 0, name
