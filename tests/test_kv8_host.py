"""Host side of the 8-bit cache's entry points, the page planner and the logits
adjustment, without a GPU: the layout of their structs, and the refusals that
return before any CUDA call (the pointers below are never dereferenced on the
host)."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from self_speculative_verification_gb300 import _build, binding as bn

OK, INVALID, UNSUPPORTED, CAPACITY, CUDA = 0, 1, 2, 4, 5
BF, F32 = bn.SPEC_BF16, bn.SPEC_F32
P = 0x1000            # 4096: aligned to 256 bytes
MIS = 0x1008          # not aligned to 16
REF = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    return bn.load_library()


@pytest.mark.parametrize("name,cls", [("spec_kv8_desc", bn.Kv8Desc), ("spec_logits_desc", bn.LogitsDesc)])
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


def cache(Hkv=2, d=128, kv=P, scales=P, batch=2, pages=8, ps=16, maxp=4, table=P):
    return bn.Kv8Desc(Hkv, d, kv, scales, batch, pages, ps, maxp, table)


BAD_CACHES = [
    (dict(Hkv=0), INVALID), (dict(pages=0), INVALID), (dict(ps=0), INVALID), (dict(ps=-16), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(ps=24), UNSUPPORTED),
    (dict(ps=8), UNSUPPORTED), (dict(ps=272), UNSUPPORTED),
    (dict(pages=1 << 30), UNSUPPORTED),                        # 2^31 (page, head) blocks
]


def attn(lib, a, c, ws=1 << 40, **ptrs):
    p = dict(q=P, kb=P, vb=P, soft_k=None, soft_v=None, seq_len=P, vis=P, row_flags=P, o=P, lse=P,
             workspace=P)
    p.update(ptrs)
    return lib.spec_verify_attn_kv8(REF(a) if a else None, p["q"], REF(c) if c else None, p["kb"], p["vb"],
                                    p["soft_k"], p["soft_v"], p["seq_len"], p["vis"], p["row_flags"],
                                    p["o"], p["lse"], p["workspace"], ws, None)


def size(lib, a, c):
    n = ctypes.c_size_t(0)
    st = lib.spec_verify_attn_kv8_workspace_size(REF(a) if a else None, REF(c) if c else None, REF(n))
    return st, n.value


def adesc(B=2, R=4, Hq=4, Hkv=2, d=128, dt=BF, n_soft=0, split=0):
    return bn.attn_desc(B, R, Hq, Hkv, d, dt, n_soft, split_tokens=split)


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_refusals(lib, dt):
    ok = adesc(dt=dt)
    for a, c, want in [
        (None, cache(), INVALID), (ok, None, INVALID),
        (adesc(B=-1, dt=dt), cache(), INVALID), (adesc(R=0, dt=dt), cache(), INVALID),
        (adesc(Hq=3, dt=dt), cache(), INVALID), (adesc(Hq=0, dt=dt), cache(), INVALID),
        (adesc(n_soft=-1, dt=dt), cache(), INVALID), (adesc(split=-64, dt=dt), cache(), INVALID),
        (adesc(split=96, dt=dt), cache(), INVALID),
        (adesc(R=257, dt=dt), cache(), UNSUPPORTED), (adesc(n_soft=65, dt=dt), cache(), UNSUPPORTED),
        (adesc(dt=7), cache(), UNSUPPORTED),
        (ok, cache(Hkv=4), INVALID), (ok, cache(d=64), INVALID), (ok, cache(batch=1), INVALID),
        (ok, cache(maxp=0), INVALID),
        (ok, cache(maxp=(1 << 26) + 1), UNSUPPORTED),          # more than 2^30 tokens a request
        (adesc(B=65536, dt=dt), cache(batch=65536), UNSUPPORTED),
        (adesc(R=256, Hq=8194, Hkv=2, dt=dt), cache(), UNSUPPORTED),   # 256 * 4097 rows a KV head
    ] + [(ok, cache(**kw), want) for kw, want in BAD_CACHES]:
        assert size(lib, a, c)[0] == want, (a and a.n_rows, c and c.page_size, want)
        assert attn(lib, a, c) == want
    st, need = size(lib, ok, cache())
    assert st == OK and need > 0
    assert lib.spec_verify_attn_kv8_workspace_size(REF(ok), REF(cache()), None) == INVALID
    assert attn(lib, ok, cache(), ws=need - 1) == CAPACITY
    for name in ("q", "kb", "vb", "seq_len", "vis", "row_flags", "o", "lse", "workspace"):
        assert attn(lib, ok, cache(), **{name: None}) == INVALID, name
    for name in ("q", "kb", "vb", "o"):
        assert attn(lib, ok, cache(), **{name: MIS}) == INVALID, name
    assert attn(lib, ok, cache(), workspace=0x1010) == INVALID          # 256-byte alignment
    for kw in (dict(kv=None), dict(kv=MIS), dict(scales=None), dict(table=None)):
        assert attn(lib, ok, cache(**kw)) == INVALID, kw
    soft = adesc(dt=dt, n_soft=4)
    assert attn(lib, soft, cache()) == INVALID                          # no soft prompt given
    assert attn(lib, soft, cache(), soft_k=P, soft_v=MIS) == INVALID
    # an empty batch is no work, whatever the pointers
    assert attn(lib, adesc(B=0, dt=dt), cache(), q=None, workspace=None, ws=0) == OK


@pytest.mark.parametrize("dt,R,Hq,d,lo,hi", [(BF, 1, 8, 128, 0, 4 << 20), (F32, 1, 8, 64, 0, 64 << 20),
                                              (BF, 256, 64, 128, 0, 1 << 30)])
def test_workspace_grows_with_the_rows_alone(lib, dt, R, Hq, d, lo, hi):
    """bf16: the workspace does not depend on the cache's capacity."""
    a = adesc(B=4, R=R, Hq=Hq, Hkv=2, d=d, dt=dt)
    small, big = cache(batch=4, d=d, maxp=4), cache(batch=4, d=d, maxp=4096)
    (s0, n0), (s1, n1) = size(lib, a, small), size(lib, a, big)
    assert s0 == s1 == OK and lo < n0 <= n1 < hi
    if dt == BF:
        assert n0 == n1
    s2, n2 = size(lib, adesc(B=8, R=R, Hq=Hq, Hkv=2, d=d, dt=dt), cache(batch=8, d=d, maxp=4))
    assert s2 == OK and n2 >= n0


def commit(lib, c, dt=BF, B=2, R=4, cap=4, n_free=8, **ptrs):
    p = dict(kb=P, vb=P, path=P, acc_len=P, seq_len=P, free_pages=P, free_head=P)
    p.update(ptrs)
    return lib.kv8_commit(REF(c) if c else None, dt, B, R, p["kb"], p["vb"], cap, p["path"], p["acc_len"],
                          p["seq_len"], p["free_pages"], n_free, p["free_head"], None)


def test_commit_refusals(lib):
    assert commit(lib, None) == INVALID
    for kw, want in BAD_CACHES + [(dict(batch=1), INVALID), (dict(maxp=0), INVALID),
                                  (dict(maxp=(1 << 26) + 1), UNSUPPORTED),
                                  (dict(kv=None), INVALID), (dict(kv=MIS), INVALID),
                                  (dict(scales=None), INVALID), (dict(table=None), INVALID)]:
        assert commit(lib, cache(**kw)) == want, kw
    for kw, want in [(dict(dt=2), UNSUPPORTED), (dict(B=-1), INVALID), (dict(R=0), INVALID),
                     (dict(cap=-1), INVALID), (dict(n_free=-1), INVALID), (dict(kb=MIS), INVALID),
                     (dict(vb=MIS), INVALID)] + [
                         ({n: None}, INVALID) for n in ("kb", "vb", "path", "acc_len", "seq_len",
                                                        "free_pages", "free_head")]:
        assert commit(lib, cache(), **kw) == want, kw
    assert commit(lib, cache(), B=0, kb=None, path=None) == OK


def append(lib, c, dt=BF, n=4, k=P, v=P, sk=256, sv=256, slots=P):
    return lib.kv8_append(REF(c) if c else None, dt, n, k, sk, v, sv, slots, None)


def test_append_refusals(lib):
    assert append(lib, None) == INVALID
    for kw, want in BAD_CACHES + [(dict(kv=None), INVALID), (dict(kv=MIS), INVALID),
                                  (dict(scales=None), INVALID)]:
        assert append(lib, cache(**kw), sk=1 << 20, sv=1 << 20) == want, kw
    for kw, want in [(dict(dt=2), UNSUPPORTED), (dict(n=-1), INVALID), (dict(k=None), INVALID),
                     (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(k=MIS), INVALID),
                     (dict(v=MIS), INVALID), (dict(sk=255), INVALID), (dict(sv=248), INVALID),
                     (dict(sk=260), INVALID),                   # 520 bytes: not 16-byte rows
                     (dict(dt=F32, sv=258), INVALID)]:
        assert append(lib, cache(), **kw) == want, kw
    # no tokens, no table: nothing to do
    assert append(lib, cache(table=None, maxp=0, batch=0), n=0, k=None, v=None, slots=None) == OK


def plan(lib, B=2, ps=16, pages=8, maxp=4, n_free=8, n_slots=4, **ptrs):
    p = dict(seq_len=P, n_new=P, table=P, free_pages=P, free_head=P, cu=P, slots=P, new_len=2 * P)
    p.update(ptrs)
    return lib.spec_page_plan(B, ps, pages, maxp, p["seq_len"], p["n_new"], p["table"], p["free_pages"],
                              n_free, p["free_head"], p["cu"], n_slots, p["slots"], p["new_len"], None)


def test_plan_refusals(lib):
    for kw, want in [(dict(B=-1), INVALID), (dict(ps=0), INVALID), (dict(pages=0), INVALID),
                     (dict(maxp=0), INVALID), (dict(n_free=-1), INVALID), (dict(n_slots=-1), INVALID),
                     (dict(cu=None), INVALID), (dict(slots=None), INVALID), (dict(free_head=None), INVALID),
                     (dict(seq_len=None), INVALID), (dict(n_new=None), INVALID), (dict(table=None), INVALID),
                     (dict(free_pages=None), INVALID), (dict(seq_len=P, new_len=P), INVALID),
                     (dict(ps=1 << 16, maxp=(1 << 14) + 1), UNSUPPORTED)]:
        assert plan(lib, **kw) == want, kw


def adjust(lib, d, **ptrs):
    names = ("logits", "out", "history", "hist_len", "n_prompt", "tokens", "tree_parent", "row_node",
             "repetition", "presence", "frequency", "bias_ids", "bias", "mask_bits", "row_mask")
    p = dict.fromkeys(names, P)
    p.update(ptrs)
    return lib.spec_logits_adjust(REF(d) if d else None, *[p[n] for n in names], None)


def test_logits_refusals(lib):
    def D(B=2, Rj=4, V=100, dt=BF, N=8, H=16, nb=4, nm=2):
        return bn.logits_desc(B, Rj, V, dt, N, H, nb, nm)

    assert adjust(lib, None) == INVALID
    for kw, want in [(dict(B=-1), INVALID), (dict(Rj=0), INVALID), (dict(V=0), INVALID),
                     (dict(N=-1), INVALID), (dict(H=-1), INVALID), (dict(nb=-1), INVALID),
                     (dict(nm=-1), INVALID), (dict(dt=2), UNSUPPORTED), (dict(N=257), UNSUPPORTED),
                     (dict(nb=1025), UNSUPPORTED), (dict(B=65536), UNSUPPORTED)]:
        assert adjust(lib, D(**kw)) == want, kw
    for n in ("logits", "out", "history", "hist_len", "tokens", "tree_parent", "bias_ids", "bias",
              "mask_bits", "row_mask"):
        assert adjust(lib, D(), **{n: None}) == INVALID, n
    assert adjust(lib, D(B=0), logits=None, out=None) == OK


def test_descriptor_of_the_wrong_tensors():
    kv = torch.zeros(4, 2, 2, 2, 8, 64, dtype=torch.uint8)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        bn.kv8_desc(kv.float(), torch.zeros(4, 2, 2))
    with pytest.raises(ValueError, match="page_size"):
        bn.kv8_desc(kv[:, :, :, :1], torch.zeros(4, 2, 2))
    with pytest.raises(TypeError, match="CUDA"):
        bn.kv8_desc(kv, torch.zeros(4, 2, 2))


def test_the_header_compiles_as_c(tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if not gcc:
        pytest.skip("no C compiler")
    src = tmp_path / "h.c"
    src.write_text('#include "specverify.h"\nint main(void) { return 0; }\n')
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", _build.INCLUDE, str(src),
                    "-o", os.devnull], check=True)
