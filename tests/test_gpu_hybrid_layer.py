"""The example's hybrid layer (SSD mixer, then attention with rotary positions over a paged cache): a
prompt in chunks followed by single tokens equals the same tokens in one prompt."""
import sys
from pathlib import Path

import pytest
import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1] / "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", [torch.int8, torch.bfloat16])
def test_chunks_and_tokens_equal_one_prompt(cache):
    from hybrid_layer import HybridLayer
    from selective_state_space_prefill_gb300 import binding as ssm

    g = torch.Generator(device="cuda").manual_seed(3)
    total = [301, 150]
    x = [torch.randn(n, 512, generator=g, device="cuda").to(torch.bfloat16) for n in total]
    whole = HybridLayer(cache=cache).prefill(x)
    parts = HybridLayer(cache=cache)
    got = [[], []]
    for a, b in (((0, 130), (0, 146)), ((130, 130), (146, 147)), ((130, 297), (147, 147))):   # an empty chunk each
        for i, y in enumerate(parts.prefill([x[0][a[0]:a[1]], x[1][b[0]:b[1]]])):
            got[i].append(y)
    # request 1 has three tokens left, request 0 four: together, then the last of request 0 as a chunk
    for t in range(3):
        y = parts.decode(torch.stack([x[0][297 + t], x[1][147 + t]]))
        got[0].append(y[:1])
        got[1].append(y[1:])
    got[0].append(parts.prefill([x[0][300:], x[1][:0]])[0])
    assert parts.lens == total and ssm.device_status() == 0
    for w, p in zip(whole, got):
        p = torch.cat(p)
        # both sides round every projection, the cache and each output to bf16 (2^-8) along two ways through
        # the same layer; the values are sums of O(1) terms
        err = (p.float() - w.float()).abs().max()
        assert float(err) <= 16 * 2.0 ** -8 * float(w.float().abs().max()) / 4, float(err)
        rel = float((p.float() - w.float()).norm() / w.float().norm())
        assert rel <= 2.0 ** -7, rel


def test_example_runs(capsys):
    import hybrid_layer
    hybrid_layer.main()
    out = capsys.readouterr().out
    assert "cached tokens [708, 137, 13]" in out and "status 0" in out
