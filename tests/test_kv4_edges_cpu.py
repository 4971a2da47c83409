"""The key/value step's host side without a GPU: what the layers pass on to the calls."""
import pytest

torch = pytest.importorskip("torch")

from bitlinear_bitnet_quant_b200 import api, chain  # noqa: E402


def _chain(**att):
    return chain.BitLinearChain([], 2, 256, 512, "cpu", attention=dict(B=2, L=1, T_cap=100, heads=2, **att))


def test_chain_passes_the_bound_on_positions(monkeypatch):
    seen = []
    monkeypatch.setattr(api, "bitnet_kv4_append", lambda *a, **kw: seen.append(("append", kw["pos"], kw["lens"])))
    monkeypatch.setattr(api, "bitnet_kv4_attention", lambda *a, **kw: seen.append(("attention", kw["pos"], kw["t_max"])))
    monkeypatch.setattr(api, "bitnet_add", lambda *a, **kw: None)
    ch = _chain(kv_bits=4)
    ch.layers = [None]
    ch.gamma_q = ch.gamma_k = [None]
    ch.kv4 = [None]
    monkeypatch.setattr(ch, "layer", lambda parts, w, stream, i: (ch.attend(i, stream), None))
    pos = torch.zeros(2, dtype=torch.int32)
    ch.forward(torch.zeros(2, 256), pos=pos, t_max=40)
    ch.forward(torch.zeros(2, 256), t0=3)
    assert seen == [("append", pos, None), ("attention", pos, 40), ("append", None, None), ("attention", None, None)]
    with pytest.raises(ValueError, match="kv_bits=4"):
        _chain().forward(torch.zeros(2, 256), t_max=10)
