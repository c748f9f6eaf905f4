"""Host-side checks of the latent-attention calls (include/kda_mla.h): what is
declared is exported, and bad arguments are refused before anything is
launched. No GPU needed: pointers are never followed."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import gated_delta_rule_chunk_amd as kda

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(16)]
HEADER = os.path.join(os.path.dirname(kda.HEADER_PATH), "kda_mla.h")
BAD, UNSUP = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_chunk_amd import _build
        _build.build()
    return kda.load_library()


def test_header_symbols_are_exported(lib):
    names = set(kda.declared_symbols(HEADER))
    assert names == {"kda_mla_fwd", "kda_mla_bwd", "kda_mla_bwd_workspace_bytes", "kda_mla_cache_append",
                     "kda_mla_step", "kda_mla_step_workspace_bytes"}
    out = subprocess.run(["nm", "-D", "--defined-only", kda.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= {line.split()[-1] for line in out.splitlines() if " T " in line}


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "kda_mla.h"\nint main(void) { return KDA_OK; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), "-c", str(src), "-o",
                    str(tmp_path / "t.o")], check=True)


def _expanded(**kw):
    a = dict(q=P[0], kv=P[1], kr=P[2], row=64, batch=6400, cuq=None, cuk=None, B=2, Tq=100, Tk=100, H=4, Dn=128, Dr=64,
             N=2, causal=1, scale=0.1, dtype=kda.KDA_BF16, rest=0)
    a.update(kw)
    return a


def _fwd(lib, o=P[3], lse=P[4], **kw):
    a = _expanded(**kw)
    return lib.kda_mla_fwd(a["q"], a["kv"], a["kr"], a["row"], a["batch"], a["cuq"], a["cuk"], a["B"], a["Tq"], a["Tk"],
                           a["H"], a["Dn"], a["Dr"], a["N"], a["causal"], a["scale"], a["dtype"], a["rest"], o, lse,
                           None)


def _bwd(lib, o=P[3], lse=P[4], d_o=P[5], ws=P[6], n=1 << 30, dq=P[7], dkv=P[8], dkr=P[9], **kw):
    a = _expanded(**kw)
    return lib.kda_mla_bwd(a["q"], a["kv"], a["kr"], a["row"], a["batch"], a["cuq"], a["cuk"], o, lse, d_o, a["B"],
                           a["Tq"], a["Tk"], a["H"], a["Dn"], a["Dr"], a["N"], a["causal"], a["scale"], a["dtype"],
                           a["rest"], ws, n, dq, dkv, dkr, None)


COMMON = [
    (dict(B=0, N=0), BAD, "B >= 1"), (dict(Tq=-1), BAD, "Tq >= 0"), (dict(Tk=-1), BAD, "Tk >= 0"),
    (dict(H=0), BAD, "H >= 1"), (dict(dtype=5), UNSUP, "dtype"), (dict(Dn=96), UNSUP, "Dn=96"),
    (dict(Dr=32), UNSUP, "Dr=32"), (dict(cuq=P[10]), BAD, "together"), (dict(cuk=P[10]), BAD, "together"),
    (dict(cuq=P[10], cuk=P[11]), BAD, "B == 1"), (dict(N=3), BAD, "N must equal B"), (dict(causal=2), BAD, "causal"),
    (dict(scale=0.0), BAD, "scale"), (dict(scale=-1.0), BAD, "scale"), (dict(scale=float("nan")), BAD, "scale"),
    (dict(scale=float("inf")), BAD, "scale"), (dict(q=None), BAD, "q must"), (dict(kv=None), BAD, "kv must"),
    (dict(kr=None), BAD, "k_rope"), (dict(Dr=0), BAD, "k_rope"), (dict(row=65), BAD, "16 bytes"),
    (dict(batch=-64), BAD, "16 bytes"), (dict(q=ctypes.c_void_p(0x10008)), BAD, "aligned"),
    (dict(Tq=1 << 30, H=1 << 10), UNSUP, "too large"),
]


@pytest.mark.parametrize("kw,status,needle", COMMON + [
    (dict(o=None), BAD, "o must"), (dict(o=P[0]), BAD, "alias q"), (dict(o=P[1]), BAD, "alias kv"),
    (dict(o=P[2]), BAD, "alias k_rope"),
])
def test_fwd_refuses(lib, kw, status, needle):
    assert _fwd(lib, **kw) == status
    assert needle in lib.kda_last_error_message().decode()


@pytest.mark.parametrize("kw,status,needle", COMMON + [
    (dict(o=None), BAD, "non-NULL"), (dict(lse=None), BAD, "non-NULL"), (dict(d_o=None), BAD, "non-NULL"),
    (dict(dq=None), BAD, "non-NULL"), (dict(dkv=None), BAD, "dkv"), (dict(dkr=None), BAD, "dk_rope"),
    (dict(kr=None, Dr=0), BAD, "dk_rope"), (dict(ws=None), BAD, "workspace"), (dict(n=16), BAD, "workspace"),
    (dict(dq=P[0]), BAD, "dq must not alias q"), (dict(dkv=P[1]), BAD, "dkv must not alias kv"),
    (dict(dkv=P[7]), BAD, "dkv must not alias dq"), (dict(ws=P[3]), BAD, "workspace must not alias o"),
    (dict(dq=ctypes.c_void_p(0x80008)), BAD, "aligned"),
])
def test_bwd_refuses(lib, kw, status, needle):
    assert _bwd(lib, **kw) == status
    assert needle in lib.kda_last_error_message().decode()


# A launch holds at most (2^32 - 1) / 256 workgroups of 256 threads. Each pair: refused, and one step below,
# which passes the check of the sizes and is refused for a missing pointer.
MOST = (2 ** 32 - 1) // 256
PACKED = dict(B=1, cuq=P[10], cuk=P[11])


@pytest.mark.parametrize("kw,less", [
    (dict(H=128, N=MOST // 128, **PACKED), dict(N=MOST // 128 - 1)),                    # (100 / 128 + N + 1) * H
    (dict(H=96, Tq=128 * 1000, N=MOST // 96 - 1000, **PACKED), dict(N=MOST // 96 - 1001)),
    (dict(H=16, B=MOST // 32 + 1, N=MOST // 32 + 1, Tq=129), dict(Tq=128)),             # B * ceil(Tq / 128) * H
    (dict(H=1, B=2 ** 31 - 1, N=2 ** 31 - 1, Tq=128 * MOST), dict(B=1, N=1)),
])
def test_fwd_refuses_more_workgroups_than_a_launch_holds(lib, kw, less):
    assert _fwd(lib, **kw) == UNSUP and "too large" in lib.kda_last_error_message().decode()
    assert _fwd(lib, o=None, **{**kw, **less}) == BAD and "o must" in lib.kda_last_error_message().decode()


@pytest.mark.parametrize("kw,less", [
    (dict(H=128, N=MOST // 128, **PACKED), dict(N=MOST // 128 - 1)),
    (dict(H=16, B=MOST // 32 + 1, N=MOST // 32 + 1, Tq=129), dict(Tq=128)),
    (dict(H=16, B=MOST // 32 + 1, N=MOST // 32 + 1, Tk=129), dict(Tk=128)),             # the keys' side alone
    (dict(H=1, B=1, N=1, Tk=MOST * 16 + 1), dict(Tk=MOST * 16)),                        # the sum of the shared key part
])
def test_bwd_refuses_more_workgroups_than_a_launch_holds(lib, kw, less):
    assert _bwd(lib, **kw) == UNSUP and "too large" in lib.kda_last_error_message().decode()
    assert _bwd(lib, dq=None, **{**kw, **less}) == BAD and "non-NULL" in lib.kda_last_error_message().decode()


def test_bwd_workspace_bytes(lib):
    w = kda.mla_bwd_workspace_bytes
    assert w(2, 100, 50, 4, 64) == 2 * 4 * 100 * 4 + 4 * 2 * 50 * 64 * 4
    assert w(1, 7, 50, 3, 0) == 96                       # 84 bytes, rounded up
    assert w(0, 1, 1, 1, 0) == w(1, -1, 1, 1, 0) == w(1, 1, 1, 1, 32) == 0


def _append(lib, **kw):
    a = dict(lat=P[0], lr=512, lb=512, kr=P[1], row=64, batch=64, cache=P[2], table=P[3], lens=P[4], cu=None, n_pages=9,
             page=16, max_pages=3, B=4, T=1, Dc=512, Dr=64, N=4, dtype=kda.KDA_BF16)
    a.update(kw)
    return lib.kda_mla_cache_append(a["lat"], a["lr"], a["lb"], a["kr"], a["row"], a["batch"], a["cache"], a["table"],
                                    a["lens"], a["cu"], a["n_pages"], a["page"], a["max_pages"], a["B"], a["T"],
                                    a["Dc"], a["Dr"], a["N"], a["dtype"], None)


CACHE = [
    (dict(dtype=9), UNSUP, "dtype"), (dict(Dc=128), UNSUP, "Dc=128"), (dict(Dr=16), UNSUP, "Dr=16"),
    (dict(page=8), UNSUP, "page_size"), (dict(page=48), UNSUP, "page_size"), (dict(n_pages=0), BAD, "n_pages"),
    (dict(max_pages=0), BAD, "max_pages"), (dict(cache=None), BAD, "non-NULL"), (dict(table=None), BAD, "non-NULL"),
    (dict(lens=None), BAD, "non-NULL"), (dict(cache=ctypes.c_void_p(0x30004)), BAD, "aligned"),
    (dict(page=1 << 20, max_pages=1 << 12), UNSUP, "2^30"), (dict(kr=None), BAD, "k_rope"), (dict(Dr=0), BAD, "k_rope"),
]


@pytest.mark.parametrize("kw,status,needle", CACHE + [
    (dict(B=-1, N=-1), BAD, "B >= 0"), (dict(N=3), BAD, "N == B"), (dict(cu=P[5], B=2), BAD, "B == 1"),
    (dict(lat=None), BAD, "latent"), (dict(lr=511), BAD, "strides"), (dict(row=3), BAD, "strides"),
    (dict(lat=P[2]), BAD, "alias"),
])
def test_append_refuses(lib, kw, status, needle):
    assert _append(lib, **kw) == status
    assert needle in lib.kda_last_error_message().decode()


def test_append_refuses_more_workgroups_than_a_launch_holds(lib):
    """A thread a chunk of 16 bytes, 72 of them a token."""
    t = MOST * 256 // 72
    assert _append(lib, B=1, N=1, T=t + 1) == UNSUP and "too large" in lib.kda_last_error_message().decode()
    assert _append(lib, B=1, N=1, T=t, lat=None) == BAD and "latent" in lib.kda_last_error_message().decode()


def _step(lib, **kw):
    a = dict(ql=P[0], ln=2048, lt=2048, lh=512, qr=P[1], rn=256, rt=256, rh=64, cache=P[2], table=P[3], lens=P[4],
             n_pages=9, page=16, max_pages=3, B=4, T=1, H=4, Dc=512, Dr=64, scale=0.1, dtype=kda.KDA_BF16, ws=P[5],
             n=1 << 30, o=P[6], lse=P[7])
    a.update(kw)
    return lib.kda_mla_step(a["ql"], a["ln"], a["lt"], a["lh"], a["qr"], a["rn"], a["rt"], a["rh"], a["cache"],
                            a["table"], a["lens"], a["n_pages"], a["page"], a["max_pages"], a["B"], a["T"], a["H"],
                            a["Dc"], a["Dr"], a["scale"], a["dtype"], a["ws"], a["n"], a["o"], a["lse"], None)


@pytest.mark.parametrize("kw,status,needle", CACHE[:12] + [
    (dict(qr=None), BAD, "q_rope"), (dict(Dr=0), BAD, "q_rope"), (dict(B=-1), BAD, "Nb >= 0"), (dict(H=0), BAD, "H >= 1"),
    (dict(T=1 << 20, H=2), BAD, "2^20"), (dict(scale=0.0), BAD, "scale"), (dict(ql=None), BAD, "q_latent"),
    (dict(lh=4), BAD, "strides"), (dict(rt=-64), BAD, "strides"), (dict(o=None), BAD, "o non-NULL"),
    (dict(o=P[0]), BAD, "alias q_latent"), (dict(o=P[2]), BAD, "alias cache"), (dict(ws=None), BAD, "workspace"),
    (dict(n=64), BAD, "workspace"), (dict(ws=P[2]), BAD, "workspace must not alias cache"),
])
def test_step_refuses(lib, kw, status, needle):
    assert _step(lib, **kw) == status
    assert needle in lib.kda_last_error_message().decode()


def test_step_refuses_more_workgroups_than_a_launch_holds(lib):
    """The join takes a workgroup a sequence at least."""
    assert _step(lib, B=MOST + 1, H=1) == UNSUP and "too large" in lib.kda_last_error_message().decode()
    assert _step(lib, B=MOST, H=1, ws=None) == BAD and "workspace" in lib.kda_last_error_message().decode()


def test_step_workspace_bytes(lib):
    w = kda.mla_step_workspace_bytes
    assert w(4, 1, 96, 512, 64, 128, torch.bfloat16) > 0
    assert w(4, 1, 96, 512, 48, 128, torch.bfloat16) == w(4, 1, 96, 128, 64, 128, torch.bfloat16) == 0
    assert w(0, 1, 96, 512, 64, 128, torch.bfloat16) == w(4, 1, 96, 512, 64, 0, torch.bfloat16) == 0


def test_empty_work_is_ok_without_launch(lib):
    assert _fwd(lib, Tq=0, q=None, o=None) == kda.KDA_OK
    assert _bwd(lib, Tq=0, Tk=0, q=None, kv=None, kr=None, dkr=None) == kda.KDA_OK
    assert _append(lib, T=0, lat=None) == kda.KDA_OK
    assert _append(lib, B=0, N=0) == kda.KDA_OK
    assert _step(lib, B=0, ql=None, ws=None) == kda.KDA_OK


def test_binding_refuses():
    q, kv, r = torch.zeros(1, 4, 2, 192), torch.zeros(1, 4, 2, 256), torch.zeros(1, 4, 64)
    with pytest.raises(ValueError, match="GPU"):
        kda.mla_fwd(q, kv, r)
    with pytest.raises(ValueError, match="must be"):
        kda.mla_fwd(q[0], kv, r)
    with pytest.raises(ValueError, match="GPU"):
        kda.mla_cache_append(torch.zeros(1, 1, 512), None, torch.zeros(1, 16, 512), torch.zeros(1, 1, dtype=torch.int32),
                             torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        kda.mla_step(torch.zeros(1, 1, 2, 512), None, torch.zeros(1, 16, 512), torch.zeros(1, 1, dtype=torch.int32),
                     torch.zeros(1, dtype=torch.int32), 1.0)


def test_declared_arguments_match_the_binding(lib):
    """One ctypes argument for each declared parameter."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name in kda.declared_symbols(HEADER):
        params = re.search(rf"\b{name}\s*\((.*?)\);", text, flags=re.S).group(1)
        assert len(getattr(lib, name).argtypes) == params.count(",") + 1, name
