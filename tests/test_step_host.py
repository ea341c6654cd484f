"""Host side of the step operators (lean_step.h), no GPU needed: the binding's
structs have the header's layout, rotary frequencies and their whole-number form
match their formulas, workspace sizes, and every argument error is found on the
host before anything could be launched."""
import ctypes
import math
import os
import re
import struct
import subprocess

import numpy as np
import pytest

from block_quantized_weight_dot_gb300 import build as lib_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lean_step.h")


@pytest.fixture(scope="module")
def lean():
    lib_build.build()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


def c_structs():
    """{struct name: [(field, kind)]} as the header declares them; kind: q (int64), d (double) or Q (pointer)."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    out = {}
    for body, name in re.findall(r"typedef struct \{(.*?)\} (\w+);", text, flags=re.S):
        fields = []
        for decl in body.split(";"):
            decl = " ".join(decl.split())
            if not decl:
                continue
            kind = "Q" if "*" in decl else "d" if decl.startswith("double") else "q"
            base = decl.replace("const ", "").split(" ", 1)[1]
            fields += [(n.strip(" *"), kind) for n in base.split(",")]
        out[name] = fields
    return out


STRUCTS = {"lean_norm_args": "_NORM", "lean_rope_args": "_ROPE", "lean_kv_pages_args": "_PAGES",
           "lean_attention_args": "_ATTENTION", "lean_logprobs_args": "_LOGPROBS"}


def test_structs_match_the_header(lean, tmp_path):
    structs = c_structs()
    assert set(structs) == set(STRUCTS)
    src = "#include <stdio.h>\n#include \"%s\"\nint main(void) {\n" % HEADER
    for name, fields in structs.items():
        src += "printf(\"%s %%zu\\n\", sizeof(%s));\n" % (name, name)
        kinds = "".join(k for _, k in fields)
        fmt = getattr(lean, STRUCTS[name]).format
        flat = re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), fmt.lstrip("<"))
        assert flat == kinds, name
    (tmp_path / "s.c").write_text(src + "return 0; }\n")
    subprocess.run(["gcc", "-o", str(tmp_path / "s"), str(tmp_path / "s.c")], check=True)
    for line in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.splitlines():
        name, size = line.split()
        assert int(size) == getattr(lean, STRUCTS[name]).size, name


class Call:
    """A struct filled by field name; pointers are small aligned numbers that nothing reads on the host."""

    def __init__(self, lean, name, fn, good):
        self.lean, self.fields, self.fn = lean, c_structs()[name], getattr(lean._lib, fn)
        self.layout, self.good = getattr(lean, STRUCTS[name]), good
        assert set(good) <= {f for f, _ in self.fields}

    def status(self, **changes):
        v = dict(self.good, **changes)
        return self.fn(self.layout.pack(*[v.get(f, 0) for f, _ in self.fields]), None)


P = 1 << 20  # stands for a device pointer, 256-byte aligned


def check_errors(call, lean, cases):
    for status, changes in cases:
        got = call.status(**changes)
        assert got == getattr(lean, "LEAN_ERR_" + status), (changes, lean.status_str(got))
    assert call.fn(None, None) == lean.LEAN_ERR_NULL


def test_norm_refusals(lean):
    call = Call(lean, "lean_norm_args", "lean_residual_norm",
                dict(rows=2, width=64, x=P, x_stride=64, h=P, h_stride=64, h_out=P, h_out_stride=64, y=P, y_stride=64,
                     w=P, eps=1e-5, res_scale=1.0))
    check_errors(call, lean, [
        ("FORMAT", dict(act_dtype=3)), ("FORMAT", dict(act_dtype=-1)), ("FORMAT", dict(act_dtype=1, res_dtype=2)),
        ("FORMAT", dict(flags=2)), ("SHAPE", dict(rows=0)), ("SHAPE", dict(width=0)), ("SHAPE", dict(x_stride=-1)),
        ("SHAPE", dict(y_stride=63)), ("SHAPE", dict(h_out_stride=0)), ("NULL", dict(x=0, h=0)),
        ("NULL", dict(h_out=0, y=0)), ("NULL", dict(x=0, post_w=P)), ("NULL", dict(x=0, gate=P)),
        ("ALIGN", dict(x=P + 2)), ("ALIGN", dict(act_dtype=1, y=P + 1)), ("ALIGN", dict(w=P + 2))])


def test_rope_refusals(lean):
    call = Call(lean, "lean_rope_args", "lean_rope_append",
                dict(n_tokens=2, n_q_heads=2, n_kv_heads=1, head_dim=64, rot_dim=64, cache_dtype=1, q=P, q_stride=128,
                     q_head_stride=64, k=P, k_stride=64, k_head_stride=64, v=P, v_stride=64, v_head_stride=64, q_out=P,
                     q_out_stride=128, q_out_head_stride=64, positions=P, slots=P, turns=P, k_cache=P, v_cache=P,
                     n_pages=4, page_size=16, page_stride=1024, place_stride=64, cache_head_stride=64, rot_scale=1.0))
    check_errors(call, lean, [
        ("FORMAT", dict(act_dtype=5)), ("FORMAT", dict(cache_dtype=0)), ("FORMAT", dict(flags=4)),
        ("SHAPE", dict(n_tokens=0)), ("SHAPE", dict(n_q_heads=-1)), ("SHAPE", dict(n_q_heads=0, n_kv_heads=0, q=0, k=0)),
        ("SHAPE", dict(head_dim=0)), ("SHAPE", dict(head_dim=65)), ("SHAPE", dict(head_dim=514)),
        ("SHAPE", dict(rot_dim=63)), ("SHAPE", dict(rot_dim=66)), ("SHAPE", dict(rot_dim=-2)),
        ("SHAPE", dict(k_stride=-1)), ("SHAPE", dict(page_stride=-8)), ("SHAPE", dict(page_size=0)),
        ("SHAPE", dict(n_pages=0)), ("SHAPE", dict(n_pages=1 << 28)), ("NULL", dict(q_out=0)), ("NULL", dict(q=0)),
        ("NULL", dict(k=0)), ("NULL", dict(v=0)), ("NULL", dict(slots=0)), ("NULL", dict(v_cache=0)),
        ("NULL", dict(k_cache=0, v_cache=0)), ("NULL", dict(positions=0)), ("NULL", dict(turns=0)),
        ("ALIGN", dict(q=P + 2)), ("ALIGN", dict(k_cache=P + 1)), ("ALIGN", dict(turns=P + 4))])


def test_pages_refusals(lean):
    call = Call(lean, "lean_kv_pages_args", "lean_kv_pages",
                dict(n_seqs=2, page_size=16, max_tokens=8, lens=P, targets=P, block_table=P, table_width=4,
                     table_stride=4, free_ring=P, ring_size=8, ring_state=P, lens_out=P + 256, ring_state_out=P + 512,
                     status=P, token_starts=P))
    check_errors(call, lean, [
        ("FORMAT", dict(flags=8)), ("SHAPE", dict(n_seqs=0)), ("SHAPE", dict(page_size=0)), ("SHAPE", dict(max_tokens=-1)),
        ("SHAPE", dict(table_width=0)), ("SHAPE", dict(table_stride=3)), ("SHAPE", dict(ring_size=0)),
        ("SHAPE", dict(max_tokens=1 << 31)), ("SHAPE", dict(n_seqs=1 << 31)), ("NULL", dict(lens=0)),
        ("NULL", dict(targets=0)), ("NULL", dict(block_table=0)), ("NULL", dict(free_ring=0)), ("NULL", dict(ring_state=0)),
        ("NULL", dict(lens_out=0)), ("NULL", dict(ring_state_out=0)), ("NULL", dict(status=0)),
        ("NULL", dict(token_starts=0)), ("ALIGN", dict(lens=P + 2)), ("ALIGN", dict(slots=P + 1))])


def test_attention_refusals(lean):
    size = lean.lean_paged_attention_workspace_bytes(2, 8, 2, 64)
    call = Call(lean, "lean_attention_args", "lean_paged_attention",
                dict(n_seqs=2, n_q_heads=8, n_kv_heads=2, head_dim=64, cache_dtype=1, q=P, q_stride=512, q_head_stride=64,
                     k_cache=P, v_cache=P, n_pages=4, page_size=16, page_stride=2048, place_stride=128,
                     cache_head_stride=64, block_table=P, table_width=2, table_stride=2, seq_lens=P, out=P, out_stride=512,
                     out_head_stride=64, scale=0.125, workspace=P, workspace_bytes=size))
    check_errors(call, lean, [
        ("FORMAT", dict(act_dtype=3)), ("FORMAT", dict(cache_dtype=0)), ("FORMAT", dict(flags=16)),
        ("SHAPE", dict(n_seqs=0)), ("SHAPE", dict(n_q_heads=7)), ("SHAPE", dict(n_kv_heads=0)), ("SHAPE", dict(head_dim=60)),
        ("SHAPE", dict(head_dim=264)), ("SHAPE", dict(head_dim=0)), ("SHAPE", dict(window=-1)), ("SHAPE", dict(n_pages=0)),
        ("SHAPE", dict(page_size=0)), ("SHAPE", dict(table_width=0)), ("SHAPE", dict(table_stride=1)),
        ("SHAPE", dict(table_width=1 << 28, table_stride=1 << 28)), ("SHAPE", dict(q_stride=-8)),
        ("SHAPE", dict(workspace_bytes=size - 1)), ("NULL", dict(q=0)), ("NULL", dict(v_cache=0)),
        ("NULL", dict(block_table=0)), ("NULL", dict(seq_lens=0)), ("NULL", dict(out=0)), ("NULL", dict(workspace=0)),
        ("ALIGN", dict(q_stride=516)), ("ALIGN", dict(q=P + 8)), ("ALIGN", dict(k_cache=P + 2)), ("ALIGN", dict(out=P + 4)),
        ("ALIGN", dict(workspace=P + 16)), ("ALIGN", dict(place_stride=132))])
    assert lean.lean_paged_attention_workspace_bytes(2, 7, 2, 64) == -1
    assert lean.lean_paged_attention_workspace_bytes(0, 8, 2, 64) == -1
    assert lean.lean_paged_attention_workspace_bytes(2, 8, 2, 20) == -1


def test_logprobs_refusals(lean):
    size = lean.lean_token_logprobs_workspace_bytes(2, 1000, 5)
    call = Call(lean, "lean_logprobs_args", "lean_token_logprobs",
                dict(rows=2, vocab=1000, logits=P, stride=1000, ids=P, scale=1.0, top_k=5, logprobs=P, ranks=P, entropy=P,
                     top_ids=P, top_logprobs=P, workspace=P, workspace_bytes=size))
    check_errors(call, lean, [
        ("FORMAT", dict(dtype=3)), ("FORMAT", dict(flags=1 << 20)), ("SHAPE", dict(rows=0)), ("SHAPE", dict(vocab=0)),
        ("SHAPE", dict(vocab=(1 << 20) + 1, stride=(1 << 20) + 1)), ("SHAPE", dict(stride=999)), ("SHAPE", dict(top_k=65)),
        ("SHAPE", dict(top_k=-1)), ("SHAPE", dict(scale=0.0)), ("SHAPE", dict(scale=-1.0)), ("SHAPE", dict(scale=math.inf)),
        ("SHAPE", dict(scale=math.nan)), ("SHAPE", dict(workspace_bytes=size - 1)), ("NULL", dict(logits=0)),
        ("NULL", dict(ids=0)), ("NULL", dict(top_ids=0)), ("NULL", dict(top_logprobs=0)), ("NULL", dict(workspace=0)),
        ("ALIGN", dict(logits=P + 2)), ("ALIGN", dict(ids=P + 1)), ("ALIGN", dict(workspace=P + 64))])
    assert lean.lean_token_logprobs_workspace_bytes(1, 1 << 21, 0) == -1


# ---- rotary frequencies ---------------------------------------------------------------

def test_frequencies_plain_linear_base(lean):
    i = np.arange(32)
    f = 10000.0 ** (-2 * i / 64)
    near = dict(rtol=1e-14, atol=0)
    np.testing.assert_allclose(lean.lean_rope_frequencies(lean.LEAN_ROPE_PLAIN, 64, 1e4), f, **near)
    np.testing.assert_allclose(lean.lean_rope_frequencies(lean.LEAN_ROPE_LINEAR, 64, 1e4, 4.0), f / 4, **near)
    base = 1e4 * 8 ** (64 / 62)
    np.testing.assert_allclose(lean.lean_rope_frequencies(lean.LEAN_ROPE_BASE, 64, 1e4, 8.0), base ** (-2 * i / 64), **near)
    # the first pair keeps its frequency, the last one is divided by the factor: what the changed base is for
    got = lean.lean_rope_frequencies(lean.LEAN_ROPE_BASE, 64, 1e4, 8.0)
    assert got[0] == 1 and abs(got[-1] * 8 / f[-1] - 1) < 1e-12


@pytest.mark.parametrize("kind", ["RAMP", "BANDS"])
@pytest.mark.parametrize("factor,trained,slow,fast", [(4.0, 4096.0, 1.0, 32.0), (8.0, 8192.0, 1.0, 4.0), (1.0, 2048.0, 1.0, 32.0)])
def test_frequencies_by_turns(lean, kind, factor, trained, slow, fast):
    """Pairs of `fast` turns or more keep their frequency, those of `slow` or fewer are divided by the factor, and
    between the two the frequency falls from the one to the other."""
    d, base = 128, 5e5
    f = base ** (-2 * np.arange(d // 2) / d)
    got = lean.lean_rope_frequencies(getattr(lean, "LEAN_ROPE_" + kind), d, base, factor, trained, slow, fast)
    turns = trained * f / (2 * math.pi)
    share = got / f
    one_more = 1 if kind == "RAMP" else 0  # its ends are rounded outwards to whole pairs
    first, last = int((turns >= fast).sum()), int((turns > slow).sum())
    np.testing.assert_allclose(share[:max(0, first - one_more)], 1, rtol=1e-12)
    np.testing.assert_allclose(share[last + one_more:], 1 / factor, rtol=1e-12)
    assert (np.diff(share) <= 1e-12).all() and (share <= 1 + 1e-12).all() and (share >= 1 / factor - 1e-12).all()
    if kind == "BANDS":
        mid = (turns < fast) & (turns > slow)
        r = (turns[mid] - slow) / (fast - slow)
        np.testing.assert_allclose(share[mid], r + (1 - r) / factor, rtol=1e-12)


def test_frequency_refusals(lean):
    f = lambda *a: lean._lib.lean_rope_frequencies(*a, ctypes.addressof((ctypes.c_double * 64)()))
    S, F = lean.LEAN_ERR_SHAPE, lean.LEAN_ERR_FORMAT
    assert f(5, 64, 1e4, 1.0, 0.0, 1.0, 2.0) == F and f(-1, 64, 1e4, 1.0, 0.0, 1.0, 2.0) == F
    assert f(0, 63, 1e4, 1.0, 0.0, 1.0, 2.0) == S and f(0, 0, 1e4, 1.0, 0.0, 1.0, 2.0) == S
    assert f(0, 64, 1.0, 1.0, 0.0, 1.0, 2.0) == S and f(1, 64, 1e4, 0.5, 0.0, 1.0, 2.0) == S
    assert f(2, 2, 1e4, 2.0, 0.0, 1.0, 2.0) == S and f(3, 64, 1e4, 2.0, 0.0, 1.0, 2.0) == S
    assert f(4, 64, 1e4, 2.0, 4096.0, 2.0, 2.0) == S and f(4, 64, math.nan, 2.0, 4096.0, 1.0, 2.0) == S
    assert lean._lib.lean_rope_frequencies(0, 64, 1e4, 1.0, 0.0, 1.0, 2.0, None) == lean.LEAN_ERR_NULL


def test_turns(lean):
    """turns / 2^64 is freq / (2 pi) to double precision, whole turns dropped; products with positions give the angle."""
    freq = np.array([0.0, 1.0, 0.5, 1e-6, 2 * math.pi * 0.25, 40.0, 3.14159, 1e-12])
    t = lean.lean_rope_turns(freq)
    assert t.dtype == np.int64
    u = [int(x) & (2 ** 64 - 1) for x in t]
    assert u[0] == 0
    for x, f in zip(u, freq):
        part = f / (2 * math.pi) - math.floor(f / (2 * math.pi))
        assert abs(x / 2 ** 64 - part) <= 2.0 ** -53 * max(1, f / 6)
    pos = 1234567
    for x, f in zip(u, freq):
        turn = (pos * x % 2 ** 64) / 2 ** 64
        assert abs(math.cos(2 * math.pi * turn) - math.cos(pos * f)) < 1e-8
    g = lean._lib.lean_rope_turns
    out = (ctypes.c_uint64 * 2)()
    for bad in (-1.0, math.inf, math.nan):
        assert g(ctypes.addressof((ctypes.c_double * 2)(0.5, bad)), 2, ctypes.addressof(out)) == lean.LEAN_ERR_SHAPE
    assert g(None, 2, ctypes.addressof(out)) == lean.LEAN_ERR_NULL
    assert g(ctypes.addressof((ctypes.c_double * 2)()), 0, ctypes.addressof(out)) == lean.LEAN_ERR_SHAPE


def test_wrapper_checks(lean):
    """Tensors of the wrong shape, type or device are refused by the binding."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        lean.lean_residual_norm(x, None, None, None, x)  # not on a GPU
    with pytest.raises(ValueError):
        lean.lean_residual_norm(torch.zeros(8), None, None, None, None)
    with pytest.raises(ValueError):
        lean.lean_token_logprobs(torch.zeros(2, 8, dtype=torch.float64), None, None)
    with pytest.raises(ValueError):
        lean.lean_kv_pages(torch.zeros(3, dtype=torch.int32), None, torch.zeros(2, 2, dtype=torch.int32), None, None, 16,
                           None, None, None, None)


def test_pages_in_place_refused(lean):
    """Results written over the inputs that other blocks still read."""
    call = Call(lean, "lean_kv_pages_args", "lean_kv_pages",
                dict(n_seqs=2, page_size=16, max_tokens=8, lens=P, targets=P + 256, block_table=P, table_width=4,
                     table_stride=4, free_ring=P, ring_size=8, ring_state=P + 512, lens_out=P + 768,
                     ring_state_out=P + 1024, status=P, token_starts=P))
    check_errors(call, lean, [("SHAPE", dict(lens_out=P)), ("SHAPE", dict(lens_out=P + 256)),
                              ("SHAPE", dict(ring_state_out=P + 512))])


def test_unit_count_limit(lean):
    """Attention over more 16-token units than 32 bits count is refused."""
    size = lean.lean_paged_attention_workspace_bytes(1 << 16, 8, 8, 64)
    call = Call(lean, "lean_attention_args", "lean_paged_attention",
                dict(n_seqs=1 << 16, n_q_heads=8, n_kv_heads=8, head_dim=64, cache_dtype=1, q=P, q_stride=512,
                     q_head_stride=64, k_cache=P, v_cache=P, n_pages=4, page_size=16, page_stride=8192, place_stride=512,
                     cache_head_stride=64, block_table=P, table_width=1 << 14, table_stride=1 << 14, seq_lens=P, out=P,
                     out_stride=512, out_head_stride=64, scale=0.125, workspace=P, workspace_bytes=size))
    check_errors(call, lean, [("SHAPE", {})])
