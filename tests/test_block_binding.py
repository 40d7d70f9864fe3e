"""What the binding of the norm with rotation and of the block-scaled FP8 cache does with arguments
that are no tensors or have too few dimensions: ValueError, as for any other that does not fit, and no
call. Without a GPU; the library is a recorder."""
import pytest
import torch

from paged_kv_cache_context_gb300 import pa


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture(params=["before CUDA", "on a device"])
def fake(request, monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(pa, "lib", lambda: rec)
    monkeypatch.setattr(pa, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(pa, "_is_device_tensor", lambda t: True)
    if request.param == "on a device":  # (a host tensor's device index is -1, and so is this one)
        monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
        monkeypatch.setattr(pa, "_raw_device", lambda: 0)
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    return rec


def arguments():
    """Every entry point with arguments that fit: (call, names of its tensors, values)."""
    q, k = torch.zeros(3, 8, 128), torch.zeros(3, 2, 128)
    tu, pos = torch.zeros(1, 64, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    w, slots = torch.ones(128), torch.zeros(3, dtype=torch.int64)
    kc, codes, sc = torch.zeros(4, 2, 32, 128), torch.zeros(4, 2, 32, 128, dtype=torch.uint8), torch.zeros(4, 2)
    bt, cu, n = (torch.zeros(s, dtype=torch.int32) for s in ((3, 4), (4,), (3,)))
    ws = torch.zeros(64, dtype=torch.uint8)
    cache = dict(k_cache=codes, v_cache=codes, k_scales=sc, v_scales=sc, block_tables=bt)
    return {
        "norm_rope": (pa.norm_rope, dict(q_out=q, k_out=k, query=q, key=k, turns=tu, positions=pos,
                                         q_weight=w, k_weight=w), {}),
        "norm_rope_and_cache": (pa.norm_rope_and_cache, dict(
            q_out=q, query=q, key=k, value=k, k_cache=kc, v_cache=kc, slot_mapping_=slots, turns=tu,
            positions=pos, q_weight=w, k_weight=w), {}),
        "append_fp8_block": (pa.append_fp8_block, dict(key=k, value=k, **cache, cu_q=cu,
                                                       context_lens=n), {}),
        "decode_fp8_block": (pa.decode_fp8_block, dict(out=q, query=q, **cache, context_lens=n,
                                                       workspace=ws), dict(num_kv_heads=2, scale=0.1)),
        "prefill_fp8_block": (pa.prefill_fp8_block, dict(
            out=q, query=q, **cache, cu_q=cu, context_lens=n, workspace=ws),
            dict(num_kv_heads=2, max_q_len=3, scale=0.1)),
    }


CASES = [(f, name) for f, (_, tensors, _) in arguments().items() for name in tensors]


@pytest.mark.parametrize("call", list(arguments()))
def test_arguments_that_fit_reach_the_library(fake, call):
    f, tensors, rest = arguments()[call]
    if not torch.cuda.is_initialized():
        with pytest.raises(ValueError, match="current device"):
            f(**tensors, **rest)
        return
    f(**tensors, **rest)
    assert [name for name, _ in fake.calls] == ["pa_" + call]


@pytest.mark.parametrize("call,name", CASES)
@pytest.mark.parametrize("what", ["nothing", "a list", "a number", "no dimensions", "one dimension",
                                  "a text"])
def test_what_is_no_tensor_or_has_no_dimensions_is_refused(fake, call, name, what):
    f, tensors, rest = arguments()[call]
    if what == "nothing" and name.endswith("_weight"):
        return  # (no norm)
    if what == "one dimension" and name == "workspace":
        return
    was = tensors[name]
    tensors[name] = {"nothing": None, "a list": [1, 2], "a number": 7, "a text": "x",
                     "no dimensions": torch.zeros((), dtype=was.dtype),
                     "one dimension": torch.zeros(5, dtype=was.dtype)}[what]
    if what == "no dimensions" and name == "workspace":
        return  # (one byte: the library refuses its size)
    with pytest.raises(ValueError):
        f(**tensors, **rest)
    assert fake.calls == []


@pytest.mark.parametrize("bad", [None, "x", [[1.0], [1.0, 2.0]], torch.ones(()), {}])
def test_frequencies_that_are_none_are_refused(bad):
    with pytest.raises(ValueError):
        pa.rope_turns(bad)
