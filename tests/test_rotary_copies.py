"""A Rotary, and the modules that hold one, copied, deep-copied and pickled: each copy points
at its own frequencies.  The GPU tests run what was copied."""
import copy
import ctypes
import pickle

import pytest

torch = pytest.importorskip("torch")


def pickled(x):
    return pickle.loads(pickle.dumps(x))


WAYS = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": pickled}


@pytest.fixture
def on_cpu(monkeypatch):
    """positions.Rotary over CPU tensors (nothing is launched)."""
    from mixed_precision_quantized_int8_amd import positions

    def dense(t, dtype, shape, device, name):
        assert t.dtype is dtype and tuple(t.shape) == shape and t.is_contiguous()
        return t.data_ptr()

    monkeypatch.setattr(positions, "_dense", dense)
    return positions


def check(a, b, shared):
    assert type(b) is type(a) and b is not a
    assert torch.equal(a.freqs, b.freqs) and (b.freqs.data_ptr() == a.freqs.data_ptr()) == shared
    assert (b.interleaved, b.factor, b.device) == (a.interleaved, a.factor, a.device)
    s = b._struct
    assert (s.freqs, s.pairs, s.interleaved) == (b.freqs.data_ptr(), a._struct.pairs, a._struct.interleaved)
    assert ctypes.c_float(b.factor).value == s.factor
    with pytest.raises(AttributeError):
        b.factor = 2.0


@pytest.mark.parametrize("way", WAYS)
def test_rotary(on_cpu, way):
    a = on_cpu.rotary(16, interleaved=True, factor=1.25, device="cpu")
    b = WAYS[way](a)
    check(a, b, shared=way == "copy")
    if way != "copy":      # its own frequencies: those of the first are not seen
        a.freqs.zero_()
        assert float(b.freqs[0]) == 1.0


def test_one_rotary_of_two_layers_stays_one(on_cpu):
    rot = on_cpu.rotary(16, device="cpu")
    a, b = copy.deepcopy([rot, {"layer": rot}])
    assert b["layer"] is a and a is not rot


@pytest.mark.parametrize("way", ["deepcopy", "pickle"])
def test_module(on_cpu, way):
    from mixed_precision_quantized_int8_amd.module import RotateHeads

    model = torch.nn.Sequential(RotateHeads(16, on_cpu.rotary(16, device="cpu"), device="cpu"),
                                RotateHeads(32, None, device="cpu"))
    got = WAYS[way](model)
    check(model[0].rotary, got[0].rotary, shared=False)
    assert got[1].rotary is None
    assert torch.equal(got[0].q_weight, model[0].q_weight)
    assert got[0].q_weight.data_ptr() != model[0].q_weight.data_ptr()


@pytest.fixture(scope="module")
def lib(i8l):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return i8l


@pytest.mark.gpu
@pytest.mark.parametrize("way", ["deepcopy", "save"])
def test_copied_modules_run(lib, way, tmp_path):
    """A copy of a training module gives the same outputs and gradients, and goes on doing so
    when the first's frequencies and memory are gone."""
    from mixed_precision_quantized_int8_amd.module import RotateHeads

    g = torch.Generator().manual_seed(1)
    model = RotateHeads(64, lib.rotary(64, interleaved=True, factor=1.5))
    q, k = (torch.randn((9, h, 64), generator=g).half().cuda() for h in (4, 1))
    pos = torch.arange(9, dtype=torch.int32, device="cuda")

    def step(m):
        a, b = q.clone().requires_grad_(), k.clone().requires_grad_()
        out = m(a, pos, b)
        return [t.detach().clone() for t in (*out, *torch.autograd.grad([o.float().square().sum() for o in out],
                                                                          (a, b, m.q_weight, m.k_weight)))]

    want = step(model)
    if way == "deepcopy":
        other = copy.deepcopy(model)
    else:
        torch.save(model, tmp_path / "model.pt")
        other = torch.load(tmp_path / "model.pt", weights_only=False)
    model.rotary.freqs.fill_(7.0)
    del model
    torch.cuda.empty_cache()
    for a, b in zip(step(other), want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_copied_decoder_layer_runs(lib):
    from mixed_precision_quantized_int8_amd.decoder import Int8DecoderLayer
    from test_decoder_gpu import D, HEADS, HIDDEN, KV, parts

    layer = Int8DecoderLayer(*parts(3), heads=HEADS, kv_heads=KV, rotary=lib.rotary(D),
                             q_norm=torch.ones(D))
    other = copy.deepcopy(layer)
    x = torch.randn((20, HIDDEN), generator=torch.Generator().manual_seed(2)).half().cuda()
    table, lens, cu = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([[1, 0]], [20], [0, 20]))
    outs = []
    for m in (layer, other):
        cache = lib.new_cache(2, 1, KV, D, page_size=16)
        outs.append(m(x, None, cache, table, lens, cu=cu))
        layer.rotary.freqs.zero_()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
