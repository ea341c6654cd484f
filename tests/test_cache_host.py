"""Host side of the caches in 8 bits and of lean_cache.h, no GPU needed: the binding's structs have the header's layout,
every argument error is found on the host before anything could be launched, and the binding refuses tensors of a wrong
shape, type or place."""
import os
import re
import subprocess

import pytest

from block_quantized_weight_dot_gb300 import build as lib_build
from test_step_binding import BF16, F32, I32, Library, Tensor, attention, rope, torch
from test_step_host import P, c_structs as step_structs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lean_cache.h")
I8 = torch.int8
STRUCTS = {"lean_kv_read_args": "_KV_READ", "lean_prefix_args": "_PREFIX"}


@pytest.fixture(scope="module")
def lean():
    lib_build.build()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


def cache_structs():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    out = {}
    for body, name in re.findall(r"typedef struct \{(.*?)\} (\w+);", text, flags=re.S):
        fields = []
        for decl in body.split(";"):
            decl = " ".join(decl.split())
            if decl:
                kind = "Q" if "*" in decl else "d" if decl.startswith("double") else "q"
                fields += [(n.strip(" *"), kind) for n in decl.replace("const ", "").split(" ", 1)[1].split(",")]
        out[name] = fields
    return out


def test_structs_match_the_header(lean, tmp_path):
    structs = cache_structs()
    assert set(structs) == set(STRUCTS)
    src = "#include <stdio.h>\n#include \"%s\"\nint main(void) {\n" % HEADER
    for name, fields in structs.items():
        src += "printf(\"%s %%zu\\n\", sizeof(%s));\n" % (name, name)
        flat = re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), getattr(lean, STRUCTS[name]).format.lstrip("<"))
        assert flat == "".join(k for _, k in fields), name
    (tmp_path / "s.c").write_text(src + "return 0; }\n")
    subprocess.run(["gcc", "-o", str(tmp_path / "s"), str(tmp_path / "s.c")], check=True)
    for line in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.splitlines():
        name, size = line.split()
        assert int(size) == getattr(lean, STRUCTS[name]).size, name


def refused(lean, fn, layout, fields, good, cases):
    call = getattr(lean._lib, fn)
    assert set(good) <= {f for f, _ in fields}
    for status, changes in cases:
        v = dict(good, **changes)
        got = call(layout.pack(*[v.get(f, 0) for f, _ in fields]), None)
        assert got == getattr(lean, "LEAN_ERR_" + status), (changes, lean.status_str(got))
    assert call(None, None) == lean.LEAN_ERR_NULL


SCALES = dict(k_scales=P, v_scales=P, scale_page_stride=16, scale_place_stride=1, scale_head_stride=16)


def test_append_refusals(lean):
    good = dict(n_tokens=2, n_q_heads=2, n_kv_heads=1, head_dim=64, rot_dim=64, cache_dtype=lean.LEAN_I8, q=P, q_stride=128,
                q_head_stride=64, k=P, k_stride=64, k_head_stride=64, v=P, v_stride=64, v_head_stride=64, q_out=P,
                q_out_stride=128, q_out_head_stride=64, positions=P, slots=P, turns=P, k_cache=P, v_cache=P, n_pages=4,
                page_size=16, page_stride=1024, place_stride=64, cache_head_stride=64, rot_scale=1.0, **SCALES)
    refused(lean, "lean_rope_append", lean._ROPE, step_structs()["lean_rope_args"], good, [
        ("NULL", dict(k_scales=0)), ("NULL", dict(v_scales=0)), ("SHAPE", dict(scale_page_stride=-1)),
        ("SHAPE", dict(scale_place_stride=-1)), ("SHAPE", dict(scale_head_stride=-16)), ("ALIGN", dict(k_scales=P + 2)),
        ("ALIGN", dict(v_scales=P + 1)), ("FORMAT", dict(act_dtype=3)), ("FORMAT", dict(cache_dtype=4)), ("NULL", dict(slots=0)),
        ("NULL", dict(v_cache=0)), ("SHAPE", dict(head_dim=65)), ("FORMAT", dict(flags=2))])


def test_attention_refusals(lean):
    size = lean.lean_paged_attention_workspace_bytes(2, 8, 2, 64)
    good = dict(n_seqs=2, n_q_heads=8, n_kv_heads=2, head_dim=64, cache_dtype=lean.LEAN_I8, q=P, q_stride=512, q_head_stride=64,
                k_cache=P, v_cache=P, n_pages=4, page_size=16, page_stride=2048, place_stride=128, cache_head_stride=64,
                block_table=P, table_width=2, table_stride=2, seq_lens=P, out=P, out_stride=512, out_head_stride=64,
                scale=0.125, workspace=P, workspace_bytes=size, **SCALES)
    refused(lean, "lean_paged_attention", lean._ATTENTION, step_structs()["lean_attention_args"], good, [
        ("NULL", dict(k_scales=0)), ("NULL", dict(v_scales=0)), ("SHAPE", dict(scale_page_stride=-1)),
        ("SHAPE", dict(scale_place_stride=-1)), ("SHAPE", dict(scale_head_stride=-16)), ("ALIGN", dict(k_scales=P + 2)),
        ("ALIGN", dict(v_scales=P + 1)), ("FORMAT", dict(act_dtype=3)), ("FORMAT", dict(cache_dtype=4)),
        ("SHAPE", dict(head_dim=72)), ("SHAPE", dict(head_dim=8)), ("ALIGN", dict(place_stride=136)),
        ("ALIGN", dict(page_stride=2056)), ("ALIGN", dict(cache_head_stride=72)), ("ALIGN", dict(v_cache=P + 8)),
        ("SHAPE", dict(workspace_bytes=size - 1))])


def test_read_refusals(lean):
    good = dict(n_tokens=3, n_kv_heads=2, head_dim=64, out_dtype=1, cache_dtype=lean.LEAN_I8, k_cache=P, v_cache=P, n_pages=4,
                page_size=16, page_stride=2048, place_stride=128, cache_head_stride=64, slots=P, k_out=P, k_out_stride=128,
                k_out_head_stride=64, v_out=P, v_out_stride=128, v_out_head_stride=64, **SCALES)
    refused(lean, "lean_kv_read", lean._KV_READ, cache_structs()["lean_kv_read_args"], good, [
        ("FORMAT", dict(out_dtype=3)), ("FORMAT", dict(cache_dtype=0)), ("FORMAT", dict(cache_dtype=4)),
        ("FORMAT", dict(flags=2)), ("SHAPE", dict(n_tokens=0)), ("SHAPE", dict(n_tokens=1 << 31)), ("SHAPE", dict(n_kv_heads=0)),
        ("SHAPE", dict(n_kv_heads=65537)), ("SHAPE", dict(head_dim=0)), ("SHAPE", dict(head_dim=513)), ("SHAPE", dict(n_pages=0)),
        ("SHAPE", dict(page_size=-1)), ("SHAPE", dict(n_pages=1 << 28)), ("SHAPE", dict(page_stride=-1)),
        ("SHAPE", dict(v_out_stride=-1)), ("SHAPE", dict(scale_head_stride=-1)), ("NULL", dict(k_cache=0, v_cache=0, k_out=0, v_out=0)),
        ("NULL", dict(k_cache=0)), ("NULL", dict(v_out=0)), ("NULL", dict(slots=0)), ("NULL", dict(k_scales=0)),
        ("NULL", dict(v_scales=0)), ("ALIGN", dict(k_out=P + 1)), ("ALIGN", dict(slots=P + 2)), ("ALIGN", dict(v_scales=P + 2)),
        ("ALIGN", dict(cache_dtype=1, k_cache=P + 1)), ("ALIGN", dict(out_dtype=0, v_out=P + 2))])


def test_prefix_refusals(lean):
    size = lean.lean_prefix_attention_workspace_bytes(4, 8, 2, 64, 2)
    good = dict(n_seqs=4, n_q_heads=8, n_kv_heads=2, head_dim=64, cache_dtype=1, q=P, q_stride=512, q_head_stride=64,
                k_cache=P, v_cache=P, n_pages=4, page_size=16, page_stride=2048, place_stride=128, cache_head_stride=64,
                n_prefixes=2, prefix_table=P, prefix_width=3, prefix_stride=3, prefix_lens=P, seq_starts=P, block_table=P,
                table_width=2, table_stride=2, seq_lens=P, out=P, out_stride=512, out_head_stride=64, scale=0.125,
                workspace=P, workspace_bytes=size)
    fields, call = cache_structs()["lean_prefix_args"], (lean, "lean_prefix_attention", lean._PREFIX)
    refused(*call, fields, good, [
        ("FORMAT", dict(act_dtype=3)), ("FORMAT", dict(cache_dtype=0)), ("FORMAT", dict(flags=2)), ("SHAPE", dict(n_seqs=0)),
        ("SHAPE", dict(n_q_heads=7)), ("SHAPE", dict(n_kv_heads=0)), ("SHAPE", dict(head_dim=60)), ("SHAPE", dict(head_dim=136)),
        ("SHAPE", dict(n_prefixes=0)), ("SHAPE", dict(n_prefixes=5)), ("SHAPE", dict(n_pages=0)), ("SHAPE", dict(page_size=0)),
        ("SHAPE", dict(prefix_width=0)), ("SHAPE", dict(prefix_stride=2)), ("SHAPE", dict(table_stride=1)),
        ("SHAPE", dict(prefix_width=1 << 28, prefix_stride=1 << 28)), ("SHAPE", dict(table_width=1 << 28, table_stride=1 << 28)),
        ("SHAPE", dict(q_stride=-8)), ("SHAPE", dict(page_stride=-8)), ("SHAPE", dict(workspace_bytes=size - 1)),
        ("NULL", dict(q=0)), ("NULL", dict(v_cache=0)), ("NULL", dict(prefix_table=0)), ("NULL", dict(prefix_lens=0)),
        ("NULL", dict(seq_starts=0)), ("NULL", dict(block_table=0)), ("NULL", dict(seq_lens=0)), ("NULL", dict(out=0)),
        ("NULL", dict(workspace=0)), ("ALIGN", dict(q_stride=516)), ("ALIGN", dict(q=P + 8)), ("ALIGN", dict(out=P + 8)),
        ("ALIGN", dict(k_cache=P + 2)), ("ALIGN", dict(place_stride=132)), ("ALIGN", dict(workspace=P + 16)),
        ("ALIGN", dict(seq_starts=P + 2)), ("ALIGN", dict(lse=P + 1))])
    refused(*call, fields, dict(good, cache_dtype=3, **SCALES), [
        ("NULL", dict(k_scales=0)), ("NULL", dict(v_scales=0)), ("SHAPE", dict(head_dim=72)), ("ALIGN", dict(place_stride=136)),
        ("SHAPE", dict(scale_place_stride=-1)), ("ALIGN", dict(v_scales=P + 2))])
    for bad in ((0, 8, 2, 64, 1), (4, 7, 2, 64, 1), (4, 8, 2, 144, 1), (4, 8, 2, 64, 0), (4, 8, 2, 64, 5), (4, 8, 2, 20, 1)):
        assert lean.lean_prefix_attention_workspace_bytes(*bad) == -1
    # own tokens in more 16-token units than 32 bits count
    big = dict(good, n_seqs=1 << 16, n_q_heads=8, n_kv_heads=8, table_width=1 << 14, table_stride=1 << 14,
               workspace_bytes=lean.lean_prefix_attention_workspace_bytes(1 << 16, 8, 8, 64, 2))
    refused(*call, fields, big, [("SHAPE", {})])


# ---- the binding, with stand-ins for tensors and for the library ----------------------------

@pytest.fixture
def binding(lean, monkeypatch):
    lean._here()
    monkeypatch.setattr(lean, "_here", lambda: 0)
    monkeypatch.setattr(lean, "_lib", Library(lean._lib))
    return lean


def in8(call):
    fn, args = call()
    cache, scales = (lambda: Tensor((3, 16, 2, 64), I8)), (lambda: Tensor((3, 16, 2), F32, stride=(32, 1, 16)))
    return fn, dict(args, k_cache=cache(), v_cache=cache(), k_scales=scales(), v_scales=scales())


def append8():
    return in8(rope)


def attention8():
    return in8(attention)


def read8():
    t = lambda: Tensor((5, 2, 64), BF16)  # noqa: E731
    fn, args = in8(lambda: ("lean_kv_read", dict(slots=Tensor((5,), I32), k_out=t(), v_out=t())))
    return fn, args


def prefix():
    cache = lambda: Tensor((3, 16, 2, 64), BF16)  # noqa: E731
    return "lean_prefix_attention", dict(q=Tensor((5, 8, 64), F32), k_cache=cache(), v_cache=cache(),
                                         prefix_table=Tensor((2, 7), I32), prefix_lens=Tensor((2,), I32),
                                         seq_starts=Tensor((3,), I32), block_table=Tensor((5, 3), I32),
                                         seq_lens=Tensor((5,), I32), out=Tensor((5, 8, 64), F32), scale=1.0,
                                         lse=Tensor((5, 8), F32), workspace=Tensor((1 << 26,), torch.uint8))


def prefix8():
    return in8(prefix)


CALLS = [append8, attention8, read8, prefix8]


@pytest.mark.parametrize("call", CALLS + [prefix])
def test_current_gpu_alone(binding, call):
    fn, args = call()
    getattr(binding, fn)(stream=0, **args)
    assert binding._lib.calls == 1
    for name, t in args.items():
        if isinstance(t, Tensor):
            for device in (-1, 1):
                with pytest.raises(ValueError, match="current GPU"):
                    getattr(binding, fn)(stream=0, **dict(args, **{name: Tensor(t.shape, t.dtype, device, t.stride())}))
    assert binding._lib.calls == 1


@pytest.mark.parametrize("call", CALLS)
def test_scales(binding, call):
    """Of the caches' pages, places and heads, both alike, and only beside caches in 8 bits."""
    fn, args = call()
    for name in ("k_scales", "v_scales"):
        for bad in (Tensor((3, 16, 2), BF16), Tensor((3, 2, 16), F32), Tensor((3, 16, 2, 1), F32), Tensor((3, 16, 2), F32)):
            with pytest.raises(ValueError, match="scales"):
                getattr(binding, fn)(stream=0, **dict(args, **{name: bad}))
    sixteen = {n: Tensor((3, 16, 2, 64), BF16) for n in ("k_cache", "v_cache")}
    with pytest.raises(ValueError, match="int8"):
        getattr(binding, fn)(stream=0, **dict(args, **sixteen))
    with pytest.raises(ValueError, match="v_cache"):
        getattr(binding, fn)(stream=0, **dict(args, v_cache=sixteen["v_cache"]))
    assert binding._lib.calls == 0


@pytest.mark.parametrize("call", CALLS)
def test_missing_scales_reach_the_library(binding, call, monkeypatch):
    fn, args = call()
    monkeypatch.setattr(binding, "_lib", binding._lib.real)
    for missing in (["k_scales"], ["v_scales"], ["k_scales", "v_scales"]):
        with pytest.raises(binding.LeanError) as e:
            getattr(binding, fn)(stream=0, **dict(args, **{n: None for n in missing}))
        assert e.value.status == binding.LEAN_ERR_NULL


def test_read_of_one_cache(binding):
    fn, args = read8()
    for half in ("k", "v"):
        rest = dict(args, **{half + n: None for n in ("_cache", "_scales", "_out")})
        getattr(binding, fn)(stream=0, **rest)
    assert binding._lib.calls == 2
    for bad in (dict(k_out=Tensor((5, 2, 32), BF16)), dict(k_out=Tensor((4, 2, 64), BF16)), dict(v_out=Tensor((5, 2, 64), F32)),
                dict(k_cache=None, k_scales=None, v_cache=None, v_scales=None), dict(slots=Tensor((5,), torch.int64)),
                dict(k_out=Tensor((5, 2, 64), torch.float64), v_out=Tensor((5, 2, 64), torch.float64)),
                dict(k_cache=Tensor((48, 2, 64), I8))):
        with pytest.raises(ValueError):
            getattr(binding, fn)(stream=0, **dict(args, **bad))
    assert binding._lib.calls == 2


def test_prefix_shapes(binding):
    fn, args = prefix()
    for bad in (dict(prefix_lens=Tensor((3,), I32)), dict(seq_starts=Tensor((2,), I32)), dict(block_table=Tensor((4, 3), I32)),
                dict(prefix_table=Tensor((14,), I32)), dict(prefix_table=Tensor((2, 7), torch.int64)), dict(seq_lens=Tensor((4,), I32)),
                dict(lse=Tensor((8, 5), F32)), dict(out=Tensor((5, 8, 64), BF16)), dict(workspace=Tensor((1 << 26,), I8)),
                dict(v_cache=Tensor((3, 16, 2, 64), BF16, stride=(4096, 128, 64, 1)))):
        with pytest.raises(ValueError):
            getattr(binding, fn)(stream=0, **dict(args, **bad))
    assert binding._lib.calls == 0
