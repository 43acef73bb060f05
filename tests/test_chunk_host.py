"""Host side of spec_rope, kv_append and the chunk attention, without a GPU: the
layout of their structs, and the refusals that return before any CUDA call (the
device pointers below are never dereferenced on the host)."""

import ctypes
import math
import os
import shutil
import subprocess

import pytest

from self_speculative_verification_gb300 import _build, binding as bn

OK, INVALID, UNSUPPORTED, CAPACITY = 0, 1, 2, 4
BF, F32 = bn.SPEC_BF16, bn.SPEC_F32
P = 0x100000          # aligned to 256 bytes
O = 0x40000000        # another place
MIS = 0x100008        # not aligned to 16
REF = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    return bn.load_library()


@pytest.mark.parametrize("name,cls", [("spec_chunk_desc", bn.ChunkDesc), ("spec_rope_desc", bn.RopeDesc)])
def test_struct_layout_matches_c(name, cls, tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if not gcc:
        pytest.skip("no C compiler")
    fields = [f[0] for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "specverify.h"\nint main(void) {\n'
                   f'printf("%zu", sizeof({name}));\n'
                   + "".join(f'printf(" %zu", offsetof({name}, {f}));\n' for f in fields)
                   + "return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-I", _build.INCLUDE, str(src), "-o", str(exe)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert out == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


def test_new_names_are_public():
    import self_speculative_verification_gb300 as pkg
    for n in ("rope_desc", "spec_rope_freqs", "spec_rope", "kv_append", "chunk_desc", "spec_chunk_attn",
              "spec_chunk_attn_workspace_size", "spec_chunk_attn_kv8", "spec_chunk_attn_kv8_workspace_size"):
        assert getattr(pkg, n) is getattr(bn, n)
    header = open(os.path.join(_build.INCLUDE, "specverify.h")).read()
    for n, v in (("SPEC_ROPE_PAIRS", 0), ("SPEC_ROPE_HALVES", 1), ("SPEC_ROPE_PLAIN", 0), ("SPEC_ROPE_LINEAR", 1),
                 ("SPEC_ROPE_RAMP", 2)):
        assert getattr(bn, n) == v and " ".join(header.split()).count(f"#define {n} {v}") == 1


# --------------------------------------------------------------- chunk attention

def rows_cache(kind=bn.SPEC_KV_PAGED, dt=BF, Hkv=2, d=128, k=P, v=P, batch=2, max_seq=64, pages=8, ps=16, maxp=4,
               table=P):
    return bn.KvDesc(kind, dt, Hkv, d, k, v, batch, max_seq, pages, ps, maxp, table)


def cache8(dt=BF, Hkv=2, d=128, k=P, scales=P, batch=2, pages=8, ps=16, maxp=4, table=P):
    return bn.Kv8Desc(Hkv, d, k, scales, batch, pages, ps, maxp, table)


def chunk(B=2, n=9, Hq=4, Hkv=2, d=128, dt=BF, scale=0.0):
    return bn.chunk_desc(B, n, Hq, Hkv, d, dt, scale)


def calls(lib, kv8):
    size_fn = lib.spec_chunk_attn_kv8_workspace_size if kv8 else lib.spec_chunk_attn_workspace_size
    fn = lib.spec_chunk_attn_kv8 if kv8 else lib.spec_chunk_attn

    def size(a, c):
        n = ctypes.c_size_t(0)
        return size_fn(REF(a) if a else None, REF(c) if c else None, REF(n)), n.value

    def run(a, c, ws=1 << 40, stride=None, **ptrs):
        p = dict(q=P, seq_len=P, cu_new=P, o=O, lse=P, workspace=P)
        p.update(ptrs)
        return fn(REF(a) if a else None, p["q"], a.n_q_heads * a.head_dim if stride is None and a else stride or 0,
                  REF(c) if c else None, p["seq_len"], p["cu_new"], p["o"], p["lse"], p["workspace"], ws, None)

    return size, run


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
def test_chunk_refusals(lib, kv8, dt):
    size, run = calls(lib, kv8)
    cache = cache8 if kv8 else rows_cache
    ok, good = chunk(dt=dt), cache(dt=dt)
    for a, c, want in [
        (None, good, INVALID), (ok, None, INVALID), (chunk(B=-1, dt=dt), good, INVALID),
        (chunk(n=-1, dt=dt), good, INVALID), (chunk(Hq=0, dt=dt), good, INVALID),
        (chunk(Hq=3, dt=dt), good, INVALID), (chunk(Hkv=0, dt=dt), good, INVALID),
        (chunk(scale=-1.0, dt=dt), good, INVALID), (chunk(scale=math.nan, dt=dt), good, INVALID),
        (chunk(scale=math.inf, dt=dt), good, INVALID),
        (chunk(dt=7), good, UNSUPPORTED), (chunk(d=96, dt=dt), cache(d=96, dt=dt), UNSUPPORTED),
        (chunk(d=256, dt=dt), cache(d=256, dt=dt), UNSUPPORTED),
        (ok, cache(Hkv=4, dt=dt), INVALID), (ok, cache(d=64, dt=dt), INVALID), (ok, cache(batch=1, dt=dt), INVALID),
        (ok, cache(maxp=0, dt=dt), INVALID), (ok, cache(ps=24, dt=dt), UNSUPPORTED), (ok, cache(ps=0, dt=dt), INVALID),
        (ok, cache(pages=0, dt=dt), INVALID), (ok, cache(maxp=(1 << 26) + 1, dt=dt), UNSUPPORTED),
        (chunk(Hq=258, dt=dt), good, UNSUPPORTED),                             # 129 heads share a key
        (ok, cache(pages=1 << 30, dt=dt), UNSUPPORTED),
        # more work than 64 bits count
        (chunk(B=2, n=2 ** 31 - 1, Hq=256, dt=dt), cache(maxp=1 << 26, dt=dt), UNSUPPORTED),
    ]:
        assert size(a, c)[0] == want, (a and a.n_tokens, want)
        assert run(a, c) == want
    st, need = size(ok, good)
    assert st == OK and 0 < need < 1 << 27
    assert size(chunk(n=1 << 20, dt=dt), cache(dt=dt, maxp=1 << 16)) == (OK, need)
    if not kv8:
        assert size(ok, rows_cache(dt=BF if dt == F32 else F32))[0] == INVALID
        assert size(ok, rows_cache(kind=2, dt=dt))[0] == INVALID
        flat = rows_cache(kind=bn.SPEC_KV_CONTIGUOUS, dt=dt, pages=0, ps=0, maxp=0, table=None)
        assert size(ok, flat)[0] == OK
        assert size(ok, rows_cache(kind=bn.SPEC_KV_CONTIGUOUS, dt=dt, max_seq=0))[0] == INVALID
        assert size(ok, rows_cache(kind=bn.SPEC_KV_CONTIGUOUS, dt=dt, max_seq=(1 << 30) + 1))[0] == UNSUPPORTED
    assert run(ok, good, ws=need - 1) == CAPACITY
    for name in ("q", "seq_len", "cu_new", "o", "lse", "workspace"):
        assert run(ok, good, **{name: None}) == INVALID, name
    for name in ("q", "o", "workspace"):
        assert run(ok, good, **{name: MIS}) == INVALID, name
    assert run(ok, good, workspace=P + 16) == INVALID
    for kw in (dict(k=None), dict(k=MIS), dict(table=None), dict(scales=None) if kv8 else dict(v=None)):
        assert run(ok, cache(dt=dt, **kw)) == INVALID, kw
    es = 2 if dt == BF else 4
    assert run(ok, good, stride=4 * 128 - 16) == INVALID and run(ok, good, stride=4 * 128 + 2) == INVALID
    # o inside the rows of q, before and behind
    width = 4 * 128 * es
    assert run(ok, good, o=P + 8 * width) == INVALID and run(ok, good, o=P - 9 * width + 16) == INVALID
    assert run(ok, good, stride=4 * 128 * 3, o=P + 24 * width) == INVALID
    # nothing to do, whatever the pointers
    for a in (chunk(B=0, dt=dt), chunk(n=0, dt=dt)):
        assert run(a, good, q=None, o=None, workspace=None, ws=0) == OK


# --------------------------------------------------------------------- kv_append

def append(lib, c, n=5, k=P, sk=256, v=P, sv=256, slots=P):
    return lib.kv_append(REF(c) if c else None, n, k, sk, v, sv, slots, None)


@pytest.mark.parametrize("dt", [BF, F32])
def test_append_refusals(lib, dt):
    good = rows_cache(dt=dt, k=O, v=O)
    flat = dict(kind=bn.SPEC_KV_CONTIGUOUS, dt=dt)
    for c, want in [(None, INVALID), (rows_cache(kind=3, dt=dt), INVALID), (rows_cache(dt=2), UNSUPPORTED),
                    (rows_cache(dt=dt, Hkv=0), INVALID), (rows_cache(dt=dt, d=96), UNSUPPORTED),
                    (rows_cache(dt=dt, pages=0), INVALID), (rows_cache(dt=dt, ps=0), INVALID),
                    (rows_cache(dt=dt, ps=40), UNSUPPORTED), (rows_cache(max_seq=0, **flat), INVALID),
                    (rows_cache(batch=0, **flat), INVALID)]:
        assert append(lib, c) == want
    assert append(lib, good, n=-1) == INVALID
    for kw in (dict(sk=255), dict(sv=0), dict(sk=-256), dict(k=None), dict(v=None), dict(slots=None), dict(k=MIS),
               dict(v=MIS), dict(sk=258), dict(sv=257)):
        assert append(lib, good, **kw) == INVALID, kw
    assert append(lib, rows_cache(dt=dt, k=None)) == INVALID and append(lib, rows_cache(dt=dt, v=MIS)) == INVALID
    assert append(lib, good, n=0, k=None, slots=None) == OK


# --------------------------------------------------------------------- spec_rope

def rope(lib, n=6, Hq=4, Hk=2, d=64, rot=64, layout=0, dt=BF, att=1.0, freqs=(0.1,) * 32, q=P, sq=1024, qo=O, sqo=1024,
         k=P + 0x10000, sk=1024, ko=O + 0x10000, sko=1024, pos=P, B=0, seq=None, cu=None, desc=True):
    f = (ctypes.c_double * len(freqs))(*freqs) if freqs is not None else None
    a = bn.rope_desc(n, Hq, Hk, d, rot, layout, dt, att)
    return lib.spec_rope(REF(a) if desc else None, f, q, sq, qo, sqo, k, sk, ko, sko, pos, B, seq, cu, None)


@pytest.mark.parametrize("dt", [BF, F32])
def test_rope_refusals(lib, dt):
    es = 2 if dt == BF else 4
    for kw in (dict(desc=False), dict(freqs=None), dict(n=-1), dict(Hq=-1), dict(Hk=-1), dict(d=0), dict(rot=0),
               dict(rot=63), dict(rot=66), dict(B=-1), dict(att=math.nan), dict(att=math.inf),
               dict(freqs=(0.1,) * 31 + (math.nan,)), dict(freqs=(math.inf,) + (0.1,) * 31), dict(sq=255),
               dict(sqo=0), dict(sk=127), dict(sko=-1024), dict(q=None), dict(qo=None), dict(k=None), dict(ko=None),
               dict(q=MIS), dict(qo=MIS), dict(k=MIS), dict(ko=MIS), dict(sq=1026), dict(sko=1025),
               dict(pos=None), dict(pos=None, B=2, seq=P), dict(pos=None, B=2, cu=P), dict(pos=None, seq=P, cu=P)):
        assert rope(lib, dt=dt, **kw) == INVALID, kw
    for kw in (dict(dt=2), dict(dt=dt, layout=2), dict(dt=dt, d=68), dict(dt=dt, d=264, sq=4096, sqo=4096),
               dict(dt=dt, Hq=65536, sq=1 << 23, sqo=1 << 23)):
        assert rope(lib, **kw) == UNSUPPORTED, kw
    # nothing to do
    assert rope(lib, dt=dt, n=0, q=None, pos=None) == OK and rope(lib, dt=dt, Hq=0, Hk=0, sq=0) == OK
    # what is written meets what is read or written (rows of 256 and 128 elements, 1024 apart)
    row = 1024 * es
    for kw in (dict(qo=P + 16), dict(qo=P, sqo=1032), dict(qo=P + 255 * es // 16 * 16), dict(qo=P - 16),
               dict(qo=P + 3 * row + 16), dict(qo=P + 5 * row), dict(ko=P), dict(ko=O), dict(qo=P + 0x10000),
               dict(ko=O + 128 * es), dict(ko=O + 1024 * es - 16), dict(qo=P + 512 * es, sqo=1040)):
        assert rope(lib, dt=dt, **kw) == INVALID, kw


def test_rope_frequencies_refusals(lib):
    out = (ctypes.c_double * 128)()
    call = lambda rot=64, base=1e4, kind=2, factor=2.0, trained=100.0, lo=1.0, hi=2.0, out=out: \
        lib.spec_rope_freqs(rot, base, kind, factor, trained, lo, hi, out)  # noqa: E731
    assert call() == OK and call(rot=256) == OK and call(kind=0, factor=math.nan, lo=3.0) == OK
    for kw in (dict(rot=0), dict(rot=-2), dict(rot=7), dict(base=0.0), dict(base=-1.0), dict(base=math.nan),
               dict(base=math.inf), dict(factor=0.0), dict(factor=-1.0), dict(factor=math.nan), dict(factor=math.inf),
               dict(kind=1, factor=0.0), dict(trained=0.0), dict(trained=math.nan), dict(trained=math.inf),
               dict(lo=2.0), dict(lo=math.nan), dict(hi=math.nan), dict(hi=math.inf), dict(lo=-math.inf), dict(out=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(rot=258), dict(kind=3), dict(kind=-1)):
        assert call(**kw) == UNSUPPORTED, kw


@pytest.mark.parametrize("G,Hkv", [(1, 1), (5, 2), (128, 1)])
def test_rows_side_by_side_do_not_meet(lib, G, Hkv):
    """Rows of a joint projection, q and k in place: passed on to the launch, which
    alone fails without a GPU."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    Hq = G * Hkv
    w = (Hq + Hkv) * 64
    st = rope(lib, Hq=Hq, Hk=Hkv, q=P, sq=w, qo=P, sqo=w, k=P + Hq * 128, sk=w, ko=P + Hq * 128, sko=w)
    assert st == 5
