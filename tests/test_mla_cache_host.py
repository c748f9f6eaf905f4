"""Host-side checks of the calls of include/kda_mla_cache.h: what is declared is exported, and bad arguments are
refused before anything is launched. No GPU needed: pointers are never followed."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import gated_delta_rule_chunk_amd as kda
from tests import mla_cache_ref as ref

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(16)]
ODD = ctypes.c_void_p(0x90008)
HEADER = os.path.join(os.path.dirname(kda.HEADER_PATH), "kda_mla_cache.h")
BAD, UNSUP = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED
MOST = (2 ** 32 - 1) // 256          # workgroups of 256 in a launch


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_chunk_amd import _build
        _build.build()
    return kda.load_library()


def test_header_symbols_are_exported(lib):
    names = set(kda.declared_symbols(HEADER))
    assert names == {"kda_mla_mx_row_bytes", "kda_mla_cache_append_mx", "kda_mla_cache_read_mx", "kda_mla_step_mx",
                     "kda_mla_step_mx_workspace_bytes", "kda_mla_weigh", "kda_mla_weigh_workspace_bytes", "kda_mla_evict",
                     "kda_mla_evict_workspace_bytes"}
    out = subprocess.run(["nm", "-D", "--defined-only", kda.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= {line.split()[-1] for line in out.splitlines() if " T " in line}
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name in names:
        params = re.search(rf"\b{name}\s*\((.*?)\);", text, flags=re.S).group(1)
        assert len(getattr(lib, name).argtypes) == params.count(",") + 1, name


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "kda_mla_cache.h"\nint main(void) { return KDA_OK; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), "-c", str(src), "-o",
                    str(tmp_path / "t.o")], check=True)


def test_row_bytes(lib):
    for (Dc, Dr, dtype), n in {(512, 64, torch.bfloat16): 400, (512, 64, torch.float32): 528, (512, 0, torch.float32): 272,
                               (256, 64, torch.bfloat16): 264, (256, 64, torch.float32): 392, (256, 0, torch.bfloat16): 136,
                               (384, 0, torch.bfloat16): 0, (512, 32, torch.bfloat16): 0}.items():
        assert kda.mla_mx_row_bytes(Dc, Dr, dtype) == n
    assert lib.kda_mla_mx_row_bytes(512, 64, 7) == 0


def _append(lib, **kw):
    a = dict(lat=P[0], lr=512, lb=512, kr=P[1], row=64, batch=64, cache=P[2], table=P[3], lens=P[4], cu=None, n_pages=9,
             page=16, max_pages=3, B=4, T=1, Dc=512, Dr=64, N=4, dtype=kda.KDA_BF16)
    a.update(kw)
    return lib.kda_mla_cache_append_mx(a["lat"], a["lr"], a["lb"], a["kr"], a["row"], a["batch"], a["cache"], a["table"],
                                       a["lens"], a["cu"], a["n_pages"], a["page"], a["max_pages"], a["B"], a["T"],
                                       a["Dc"], a["Dr"], a["N"], a["dtype"], None)


def _read(lib, **kw):
    a = dict(cache=P[2], table=P[3], starts=None, cu=P[4], n_pages=9, page=16, max_pages=3, T=5, Dc=512, Dr=64, N=4,
             dtype=kda.KDA_BF16, rest=0, lat=P[5], kr=P[6])
    a.update(kw)
    return lib.kda_mla_cache_read_mx(a["cache"], a["table"], a["starts"], a["cu"], a["n_pages"], a["page"],
                                     a["max_pages"], a["T"], a["Dc"], a["Dr"], a["N"], a["dtype"], a["rest"], a["lat"],
                                     a["kr"], None)


STEP = dict(ql=P[0], ln=2048, lt=2048, lh=512, qr=P[1], rn=256, rt=256, rh=64, cache=P[2], table=P[3], lens=P[4],
            n_pages=9, page=16, max_pages=3, B=4, T=1, H=4, Dc=512, Dr=64, scale=0.1, dtype=kda.KDA_BF16)


def _step(lib, ws=P[5], n=1 << 30, o=P[6], lse=P[7], **kw):
    a = {**STEP, **kw}
    return lib.kda_mla_step_mx(a["ql"], a["ln"], a["lt"], a["lh"], a["qr"], a["rn"], a["rt"], a["rh"], a["cache"],
                               a["table"], a["lens"], a["n_pages"], a["page"], a["max_pages"], a["B"], a["T"], a["H"],
                               a["Dc"], a["Dr"], a["scale"], a["dtype"], ws, n, o, lse, None)


def _weigh(lib, lse=P[5], w=P[6], fresh=1, decay=1.0, form=1, out=P[7], ws=None, n=0, **kw):
    a = {**STEP, **kw}
    return lib.kda_mla_weigh(a["ql"], a["ln"], a["lt"], a["lh"], a["qr"], a["rn"], a["rt"], a["rh"], a["cache"],
                             a["table"], a["lens"], lse, w, fresh, decay, a["n_pages"], a["page"], a["max_pages"],
                             a["B"], a["T"], a["H"], a["Dc"], a["Dr"], a["scale"], a["dtype"], form, ws, n, out, None)


def _evict(lib, **kw):
    a = dict(cache=P[2], table=P[3], lens=P[4], w=P[5], keep=32, first=0, recent=0, n_pages=9, page=16, max_pages=3, B=4,
             Dc=512, Dr=64, dtype=kda.KDA_BF16, form=0, ws=P[6], n=1 << 30, tout=P[7], lout=P[8], wout=P[9])
    a.update(kw)
    return lib.kda_mla_evict(a["cache"], a["table"], a["lens"], a["w"], a["keep"], a["first"], a["recent"], a["n_pages"],
                             a["page"], a["max_pages"], a["B"], a["Dc"], a["Dr"], a["dtype"], a["form"], a["ws"], a["n"],
                             a["tout"], a["lout"], a["wout"], None)


CACHE = [
    (dict(dtype=9), UNSUP, "dtype"), (dict(Dc=128), UNSUP, "Dc=128"), (dict(Dr=16), UNSUP, "Dr=16"),
    (dict(page=8), UNSUP, "page_size"), (dict(page=48), UNSUP, "page_size"), (dict(n_pages=0), BAD, "n_pages"),
    (dict(max_pages=0), BAD, "max_pages"), (dict(cache=None), BAD, "non-NULL"), (dict(table=None), BAD, "non-NULL"),
    (dict(cache=ODD), BAD, "aligned"), (dict(page=1 << 20, max_pages=1 << 12), UNSUP, "2^30"),
]
LENS = [(dict(lens=None), BAD, "non-NULL")]
QUERIES = CACHE + LENS + [
    (dict(qr=None), BAD, "q_rope"), (dict(Dr=0), BAD, "q_rope"), (dict(B=-1), BAD, "Nb >= 0"), (dict(H=0), BAD, "H >= 1"),
    (dict(T=1 << 20, H=2), BAD, "2^20"), (dict(scale=0.0), BAD, "scale"), (dict(scale=float("nan")), BAD, "scale"),
    (dict(ql=None), BAD, "q_latent"), (dict(lh=4), BAD, "strides"), (dict(rt=-64), BAD, "strides"),
    (dict(ql=ODD), BAD, "aligned"),
]


@pytest.mark.parametrize("kw,status,needle", CACHE + LENS + [
    (dict(kr=None), BAD, "k_rope"), (dict(Dr=0), BAD, "k_rope"), (dict(B=-1, N=-1), BAD, "B >= 0"),
    (dict(N=3), BAD, "N == B"), (dict(cu=P[5], B=2), BAD, "B == 1"), (dict(lat=None), BAD, "latent"),
    (dict(lr=511), BAD, "strides"), (dict(row=3), BAD, "strides"), (dict(lat=P[2]), BAD, "alias"),
    (dict(B=1, N=1, T=MOST * 256 // 72 + 1), UNSUP, "too large"),
])
def test_append_refuses(lib, kw, status, needle):
    assert _append(lib, **kw) == status
    assert needle in lib.kda_last_error_message().decode()


@pytest.mark.parametrize("kw,status,needle", CACHE + [
    (dict(cu=None), BAD, "non-NULL"), (dict(T=-1), BAD, "T >= 0"), (dict(N=0), BAD, "N >= 1"), (dict(lat=None), BAD, "latent"),
    (dict(kr=None), BAD, "k_rope"), (dict(Dr=0), BAD, "k_rope"), (dict(lat=ODD), BAD, "aligned"), (dict(kr=ODD), BAD, "aligned"),
    (dict(lat=P[2]), BAD, "alias cache"), (dict(kr=P[5]), BAD, "alias latent"),
    (dict(T=MOST * 256 // 80 + 1), UNSUP, "too large"),
])
def test_read_refuses(lib, kw, status, needle):
    assert _read(lib, **kw) == status
    assert needle in lib.kda_last_error_message().decode()


@pytest.mark.parametrize("kw,status,needle", QUERIES + [
    (dict(o=None), BAD, "o non-NULL"), (dict(o=P[0]), BAD, "alias q_latent"), (dict(o=P[2]), BAD, "alias cache"),
    (dict(ws=None), BAD, "workspace"), (dict(n=64), BAD, "workspace"), (dict(ws=P[2]), BAD, "workspace must not alias cache"),
    (dict(B=MOST + 1, H=1), UNSUP, "too large"),
])
def test_step_refuses(lib, kw, status, needle):
    assert _step(lib, **kw) == status
    assert needle in lib.kda_last_error_message().decode()


@pytest.mark.parametrize("kw,status,needle", QUERIES + [
    (dict(lse=None), BAD, "lse"), (dict(w=None), BAD, "weights"), (dict(out=None), BAD, "weights_out"),
    (dict(fresh=-1), BAD, "fresh"), (dict(decay=-0.1), BAD, "decay"), (dict(decay=1.5), BAD, "decay"),
    (dict(decay=float("nan")), BAD, "decay"), (dict(form=2), BAD, "form"), (dict(out=P[2]), BAD, "alias cache"),
    (dict(out=P[5]), BAD, "alias lse"), (dict(out=P[0]), BAD, "alias q_latent"),
    (dict(H=129), BAD, "workspace"), (dict(H=129, ws=P[8], n=1000), BAD, "workspace"), (dict(H=129, ws=ODD, n=1 << 30), BAD, "workspace"),
    (dict(H=129, ws=P[7], n=1 << 30), BAD, "workspace must not alias weights_out"),
    (dict(H=129, ws=P[5], n=1 << 30), BAD, "workspace must not alias lse"),
])
def test_weigh_refuses(lib, kw, status, needle):
    assert _weigh(lib, **kw) == status
    assert needle in lib.kda_last_error_message().decode()


@pytest.mark.parametrize("kw,status,needle", CACHE + LENS + [
    (dict(B=-1), BAD, "Nb"), (dict(B=1 << 22), BAD, "Nb"), (dict(B=8192, max_pages=1 << 16, page=64), UNSUP, "too large"),
    (dict(form=-1), BAD, "form"), (dict(keep=-1), BAD, "keep"),
    (dict(first=-1), BAD, "first"), (dict(recent=-1), BAD, "recent"), (dict(w=None), BAD, "weights"),
    (dict(tout=None), BAD, "outputs"), (dict(lout=None), BAD, "outputs"), (dict(wout=None), BAD, "outputs"),
    (dict(ws=None), BAD, "workspace"), (dict(n=100), BAD, "workspace"), (dict(ws=ODD), BAD, "workspace"),
    (dict(wout=P[2]), BAD, "alias cache"), (dict(tout=P[4]), BAD, "alias seq_lens"), (dict(lout=P[3]), BAD, "alias page_table"),
    (dict(wout=P[3]), BAD, "alias page_table"), (dict(lout=P[7]), BAD, "alias page_table_out"),
    (dict(ws=P[5]), BAD, "workspace must not alias weights"),
])
def test_evict_refuses(lib, kw, status, needle):
    assert _evict(lib, **kw) == status
    assert needle in lib.kda_last_error_message().decode()


def test_workspace_bytes(lib):
    w = kda.mla_step_mx_workspace_bytes
    assert w(4, 1, 96, 512, 64, 128, torch.bfloat16) > 0
    assert w(4, 1, 96, 512, 48, 128, torch.bfloat16) == w(4, 1, 96, 128, 64, 128, torch.bfloat16) == 0
    assert w(0, 1, 96, 512, 64, 128, torch.bfloat16) == w(4, 1, 96, 512, 64, 0, torch.bfloat16) == 0
    g = kda.mla_weigh_workspace_bytes
    assert g(4, 1, 128, 512, 64, torch.bfloat16, 1) == g(4, 3, 96, 512, 64, torch.bfloat16, 0) == 0
    assert g(4, 3, 96, 512, 64, torch.float32, 1) == g(4, 3, 96, 384, 64, torch.bfloat16, 1) == 0
    assert g(4, 3, 96, 512, 64, torch.bfloat16, 1) >= 4 * 18 * 16 * 1088
    e = kda.mla_evict_workspace_bytes
    assert e(1, 16, 1) > 0 and e(100, 64, 128) >= 100 * 64 * 64 * 3 * 4
    assert e(0, 16, 1) == e(1, 24, 1) == e(1, 16, 0) == e(1, 1 << 20, 1 << 12) == 0


def test_empty_work_is_ok_without_launch(lib):
    assert _append(lib, T=0, lat=None) == _append(lib, B=0, N=0) == kda.KDA_OK
    assert _read(lib, T=0, lat=None) == kda.KDA_OK
    assert _step(lib, B=0, ql=None, ws=None) == _step(lib, T=0, ql=None) == kda.KDA_OK
    assert _weigh(lib, B=0, ql=None) == _weigh(lib, T=0, w=None) == kda.KDA_OK
    assert _evict(lib, B=0, cache=None) == kda.KDA_OK


def test_binding_refuses():
    i32 = torch.int32
    table, n = torch.zeros(1, 1, dtype=i32), torch.zeros(1, dtype=i32)
    cache = kda.mla_cache_mx(1, 16, 512, 0, torch.bfloat16, device="cpu")
    assert tuple(cache.shape) == (1, 16, 272) and not cache.any()
    with pytest.raises(ValueError, match="no 4-bit cache"):
        kda.mla_cache_mx(1, 16, 384, 0, torch.bfloat16, device="cpu")
    with pytest.raises(ValueError, match="no 4-bit cache"):
        kda.mla_cache_mx(1, 16, 512, 0, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        kda.mla_cache_append_mx(torch.zeros(1, 1, 512), None, cache, table, n)
    with pytest.raises(ValueError, match="GPU"):
        kda.mla_cache_read_mx(cache, table, torch.zeros(2, dtype=i32), 0, 512, torch.bfloat16)
    with pytest.raises(TypeError, match="dtype"):
        kda.mla_cache_read_mx(cache, table, torch.zeros(2, dtype=i32), 0, 512, torch.float16)
    q = torch.zeros(1, 1, 2, 512)
    with pytest.raises(ValueError, match="GPU"):
        kda.mla_step_mx(q, None, cache, table, n, 1.0)
    with pytest.raises(ValueError, match="GPU"):
        kda.mla_weigh(q, None, cache, table, n, torch.zeros(1, 1, 2), 1.0, torch.zeros(1, 16))
    with pytest.raises(ValueError, match="GPU"):
        kda.mla_evict(cache, table, n, torch.zeros(1, 16), 4)


def test_reference_rounding():
    """The oracle itself: no value off by more than 2^e, scale byte minimal, values come back."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(64, 256, generator=g) * torch.exp2(torch.randint(-90, 90, (64, 1), generator=g).float())
    c, s = ref.encode(x)
    v = ref.values(c, s)
    two = ref.power(s.long() - 127)
    assert ((v - x.double()).abs() <= two.repeat_interleave(32, 1)).all()
    a = x.double().abs().unflatten(1, (-1, 32)).amax(-1)
    assert (a <= 7 * two).all() and (a > 3.5 * two).all()
    again = ref.encode(v)
    assert torch.equal(ref.values(*again), v)
