"""The binding's own checks of the step operators' tensors, no GPU needed: with
stand-ins for tensors and for the library, a call goes through when everything is
on the current GPU, and is a ValueError when any one tensor is on the host or on
another GPU, of another type, or strided where it may not be."""
import pytest

from block_quantized_weight_dot_gb300 import build as lib_build

torch = pytest.importorskip("torch")
F32, BF16, I32, I64, U8 = torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8


class Tensor:
    """What the binding looks at of a tensor on GPU `device` (-1: the host)."""

    def __init__(self, shape, dtype, device=0, stride=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, "cuda:%d" % device if device >= 0 else "cpu"
        self._device, self._at = device, 1 << 20
        dense = [1]
        for n in reversed(shape[1:]):
            dense.insert(0, dense[0] * n)
        self._stride, self._dense = tuple(stride or dense), stride is None or tuple(stride) == tuple(dense)
        self.is_cuda = device >= 0

    def get_device(self):
        return self._device

    def stride(self):
        return self._stride

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return self._dense

    def data_ptr(self):
        return self._at

    def reshape(self, *shape):
        assert shape == (1, -1)
        return Tensor((1, self.numel()), self.dtype, self._device)


class Library:
    """Counts the calls that reach it."""

    def __init__(self, real):
        self.calls, self.real = 0, real

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def lean(monkeypatch):
    lib_build.build()
    from block_quantized_weight_dot_gb300 import lean as L
    L._here()
    monkeypatch.setattr(L, "_here", lambda: 0)
    monkeypatch.setattr(L, "_lib", Library(L._lib))
    return L


def norm():
    t = lambda *s: Tensor(s, BF16)
    return "lean_residual_norm", dict(x=t(4, 64), h=Tensor((4, 64), F32), w=Tensor((64,), F32), h_out=Tensor((4, 64), F32),
                                      y=t(4, 64), post_w=Tensor((64,), F32), gate=t(4, 64))


def rope():
    t = lambda h: Tensor((4, h, 64), F32)
    cache = lambda: Tensor((3, 16, 2, 64), BF16)
    return "lean_rope_append", dict(q=t(8), k=t(2), v=t(2), positions=Tensor((4,), I32), slots=Tensor((4,), I32),
                                    turns=Tensor((32,), I64), q_out=t(8), k_cache=cache(), v_cache=cache(), rot_dim=64,
                                    k_out=t(2))


def pages():
    t = lambda *s: Tensor(s, I32)
    return "lean_kv_pages", dict(lens=t(5), targets=t(5), block_table=t(5, 3), free_ring=t(20), ring_state=t(2),
                                 page_size=16, lens_out=t(5), ring_state_out=t(2), status=t(5), token_starts=t(6),
                                 slots=t(9), positions=t(9), token_seqs=t(9))


def attention():
    cache = lambda: Tensor((3, 16, 2, 64), BF16)
    return "lean_paged_attention", dict(q=Tensor((5, 8, 64), F32), k_cache=cache(), v_cache=cache(),
                                        block_table=Tensor((5, 3), I32), seq_lens=Tensor((5,), I32),
                                        out=Tensor((5, 8, 64), F32), scale=1.0, lse=Tensor((5, 8), F32),
                                        workspace=Tensor((1 << 22,), U8))


def logprobs():
    return "lean_token_logprobs", dict(logits=Tensor((5, 100), BF16), ids=Tensor((5,), I32), logprobs=Tensor((5,), F32),
                                       ranks=Tensor((5,), I32), entropy=Tensor((5,), F32), top_ids=Tensor((5, 3), I32),
                                       top_logprobs=Tensor((5, 3), F32), workspace=Tensor((1 << 22,), U8))


CALLS = [norm, rope, pages, attention, logprobs]


@pytest.mark.parametrize("call", CALLS)
def test_current_gpu_alone(lean, call):
    fn, args = call()
    getattr(lean, fn)(stream=0, **args)
    assert lean._lib.calls == 1
    for name, t in args.items():
        if not isinstance(t, Tensor):
            continue
        for device in (-1, 1):
            with pytest.raises(ValueError, match="current GPU"):
                getattr(lean, fn)(stream=0, **dict(args, **{name: Tensor(t.shape, t.dtype, device)}))
    assert lean._lib.calls == 1


@pytest.mark.parametrize("call", [attention, logprobs])
def test_workspace(lean, call):
    """Bytes without gaps: not another type, not every other byte of a longer buffer."""
    fn, args = call()
    for bad in (Tensor((1 << 22,), F32), Tensor((1 << 22,), torch.int8), Tensor((1 << 22,), U8, stride=(2,)),
                Tensor((1 << 22,), U8, -1), Tensor((1024, 4096), U8, stride=(8192, 1))):
        with pytest.raises(ValueError, match="workspace"):
            getattr(lean, fn)(stream=0, **dict(args, workspace=bad))
    assert lean._lib.calls == 0
    getattr(lean, fn)(stream=0, **dict(args, workspace=Tensor((1024, 4096), U8)))
    assert lean._lib.calls == 1


def test_one_cache_alone(lean, monkeypatch):
    """k_cache or v_cache without the other reaches the library, which refuses it; nothing is dropped on the way."""
    monkeypatch.setattr(lean, "_lib", lean._lib.real)
    fn, args = rope()
    for missing in ("k_cache", "v_cache"):
        for k_out in (args["k_out"], None):
            with pytest.raises(lean.LeanError) as e:
                lean.lean_rope_append(stream=0, **dict(args, k_out=k_out, **{missing: None}))
            assert e.value.status == lean.LEAN_ERR_NULL


@pytest.mark.parametrize("call,name", [(attention, "lse"), (logprobs, "top_ids"), (logprobs, "top_logprobs")])
def test_rows_first(lean, call, name):
    """Outputs with a value or more for each row: rows are the first dimension, whatever the number of elements is."""
    fn, args = call()
    rows, k = args[name].shape
    for shape in ((k, rows), (rows * k, 1), (rows, k, 1), (1, rows * k), (rows, k + 1)):
        with pytest.raises(ValueError, match=name if name != "top_ids" else "top_"):
            getattr(lean, fn)(stream=0, **dict(args, **{name: Tensor(shape, args[name].dtype)}))
    assert lean._lib.calls == 0


def test_no_rows(lean, monkeypatch):
    """No rows at all: the library's answer, as for the other sizes that it refuses."""
    monkeypatch.setattr(lean, "_lib", lean._lib.real)
    with pytest.raises(lean.LeanError) as e:
        lean.lean_token_logprobs(Tensor((0, 100), BF16), None, None, top_ids=Tensor((0, 3), I32),
                                 top_logprobs=Tensor((0, 3), F32), workspace=Tensor((1 << 22,), U8), stream=0)
    assert e.value.status == lean.LEAN_ERR_SHAPE


def test_most_sequences(lean):
    """Page bookkeeping counts chunks of sequences in 32 bits: 2^30 of them are refused, on the host."""
    lib, P = lean._lib.real, 1 << 20
    for n in (1 << 30, (1 << 31) - 600, (1 << 31) - 2):
        args = lean._PAGES.pack(n, 16, 8, P, P, P, 4, 4, P, 8, P, P + 256, P + 512, P, P, 0, 0, 0, 0)
        assert lib.lean_kv_pages(args, None) == lean.LEAN_ERR_SHAPE, n
