"""Host side of the gated and the serving libraries' C ABIs, without a GPU: the
exported symbols, the structs' layout, the sizes and every refused argument."""
import ctypes
import os
import re
import subprocess

import pytest

from selective_state_space_26_b200 import _lib, build

INC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
GATED, SERVE = os.path.join(INC, "jamba_ssm_gated.h"), os.path.join(INC, "jamba_ssm_serve.h")
P0 = 1 << 20  # addresses far apart that are never read: every case stops on the host
INV, UNS, MIS, WSP = (_lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_MISALIGNED,
                      _lib.ERR_WORKSPACE)


@pytest.fixture(scope="module")
def libs():
    build.build()
    return _lib.gated_lib(), _lib.serve_lib()


@pytest.mark.parametrize("header,names,path", [
    (GATED, _lib.GATED_EXPORTS, _lib.GATED_LIB_PATH),
    (SERVE, _lib.SERVE_EXPORTS, _lib.SERVE_LIB_PATH)])
def test_declared_symbols_are_the_exported_ones(libs, header, names, path):
    text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    declared = set(re.findall(r"\b(jamba_ssm_[a-z0-9_]+)\s*\(", text))
    assert declared == set(names)
    out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert declared <= exported
    assert not [e for e in exported if "jssm" in e], "internal symbols exported"


def test_struct_layouts_and_constants_match_the_headers(tmp_path):
    fields = {"jamba_ssm_gated_scan_params": _lib.GatedScanParams,
              "jamba_ssm_gated_scan_bwd_params": _lib.GatedScanBwdParams,
              "jamba_ssm_gated_state_update_params": _lib.GatedStateUpdateParams,
              "jamba_ssm_i8_quant_params": _lib.I8QuantParams,
              "jamba_ssm_i8_proj_params": _lib.I8ProjParams,
              "jamba_ssm_batch_maps_params": _lib.BatchMapsParams}
    lines = ['#include <stdio.h>', '#include "jamba_ssm_gated.h"', '#include "jamba_ssm_serve.h"',
             "int main(void) {", 'printf("k %d\\n", JAMBA_SSM_I8_MAX_K);',
             'printf("c %d\\n", JAMBA_SSM_GATED_CKPT_STEPS);',
             'printf("p %d %d\\n", (int)JAMBA_SSM_I8_PITCH(16), (int)JAMBA_SSM_I8_PITCH(17));']
    for name, cls in fields.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines) + "return 0; }")
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", INC, "-o", str(exe), str(src)], check=True)
    rows = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    assert rows[0] == f"k {_lib.I8_MAX_K}" and rows[1] == f"c {_lib.GATED_CKPT_STEPS}"
    assert rows[2] == "p 16 32"
    for row in filter(None, rows[3:]):
        name, f, v = row.split()
        cls = fields[name]
        assert (ctypes.sizeof(cls) if f == "size" else getattr(cls, f).offset) == int(v), row


def test_versions(libs):
    assert libs[0].jamba_ssm_gated_abi_version() == 1
    assert libs[1].jamba_ssm_serve_abi_version() == 1


def _call(fn, cls, base, **kw):
    p = cls(**{**base, **kw})
    if "struct_size" not in kw:
        p.struct_size = ctypes.sizeof(cls)
    return fn(ctypes.byref(p), None)


def _at(n):
    return P0 + (n << 34)


SCAN = dict(batch=2, seqlen=100, d_inner=64, io_dtype=_lib.BF16, x=_at(1), g=_at(2), z=_at(3),
            rate=_at(4), bias=_at(5), h0=_at(6), out=_at(7), h_final=_at(8), ckpt=_at(9))


@pytest.mark.parametrize("kw,expect", [
    (dict(struct_size=8), INV), (dict(batch=-1), INV), (dict(seqlen=-1), INV),
    (dict(d_inner=0), INV), (dict(reserved=1), INV), (dict(io_dtype=2), INV),
    (dict(x=None), INV), (dict(g=None), INV), (dict(out=None), INV),
    (dict(x_stride=63), INV), (dict(g_stride=-1), INV), (dict(z_stride=1), INV),
    (dict(x_stride=(1 << 31) + 1), UNS), (dict(d_inner=(1 << 20) + 1), UNS),
    (dict(batch=(1 << 24) + 1), UNS), (dict(batch=1 << 12, seqlen=1 << 20), UNS),
    (dict(seqlen=1 << 40), UNS), (dict(cu_seqlens=_at(10), total_tokens=-1), INV),
    (dict(cu_seqlens=_at(10), total_tokens=1 << 31), UNS),
    (dict(state_indices=_at(10)), INV), (dict(state_indices=_at(10), num_slots=1 << 31), UNS),
    (dict(initial_indices=_at(10)), INV), (dict(initial_indices=_at(10), num_slots=4), INV),
    (dict(x=_at(1) + 1), MIS), (dict(out=_at(7) + 1), MIS), (dict(rate=_at(4) + 2), MIS),
    (dict(ckpt=_at(9) + 8), MIS), (dict(h_final=_at(8) + 2), MIS),
    (dict(cu_seqlens=_at(10) + 2, total_tokens=5), MIS),
    (dict(state_indices=_at(10) + 1, num_slots=4), MIS),
    (dict(workspace=_at(11) + 8, workspace_bytes=16), MIS),
    (dict(workspace=_at(11), workspace_bytes=15), WSP),
    (dict(out=_at(1)), INV), (dict(out=_at(2) + 200 * 64 * 2 - 2), INV),
    (dict(h_final=_at(6) + 4), INV), (dict(h_final=_at(4)), INV), (dict(ckpt=_at(7)), INV),
    (dict(out=_at(5)), INV), (dict(h_final=_at(7)), INV),
    # x's rows end inside out though its first row does not
    (dict(x=_at(7) - 1000 * 128, x_stride=1000), INV),
])
def test_scan_refusals(libs, kw, expect):
    assert _call(libs[0].jamba_ssm_gated_scan, _lib.GatedScanParams, SCAN, **kw) == expect


def test_scan_accepts_up_to_the_device(libs):
    if _has_gpu():
        pytest.skip("the addresses are not real: only without a GPU")
    f, c = libs[0].jamba_ssm_gated_scan, _lib.GatedScanParams
    for kw in ({}, dict(z=None), dict(rate=None, bias=None, h0=None, h_final=None, ckpt=None),
               dict(h_final=_at(6)), dict(d_inner=1), dict(x_stride=200, g_stride=65),
               dict(cu_seqlens=_at(10), total_tokens=7), dict(seqlen=0, x=None, g=None, out=None),
               dict(state_indices=_at(10), initial_indices=_at(11), num_slots=3)):
        assert _call(f, c, SCAN, **kw) == _lib.ERR_NO_DEVICE, kw
    assert _call(f, c, SCAN, batch=0, x=None) == _lib.OK
    assert f(None, None) == INV


def _has_gpu():
    import torch
    return torch.cuda.is_available()


BWD = dict(batch=2, seqlen=100, d_inner=64, io_dtype=_lib.F32, x=_at(1), g=_at(2), z=_at(3),
           rate=_at(4), bias=_at(5), h0=_at(6), dout=_at(7), dh_final=_at(8), dx=_at(9),
           dg=_at(10), dz=_at(11), drate=_at(12), dbias=_at(13), dh0=_at(14), ckpt=_at(15),
           workspace=_at(16), workspace_bytes=1 << 30)


@pytest.mark.parametrize("kw,expect", [
    (dict(struct_size=0), INV), (dict(batch=-2), INV), (dict(io_dtype=-1), INV),
    (dict(dout=None), INV), (dict(dx=None), INV), (dict(dg=None), INV), (dict(dz=None), INV),
    (dict(z=None), INV), (dict(workspace=None), WSP), (dict(workspace_bytes=100), WSP),
    (dict(workspace=_at(16) + 4), MIS), (dict(dout=_at(7) + 2), MIS), (dict(dh0=_at(14) + 1), MIS),
    (dict(dx=_at(10)), INV), (dict(dx=_at(7)), INV), (dict(dh0=_at(8)), INV),
    (dict(drate=_at(13)), INV), (dict(dg=_at(2)), INV), (dict(workspace=_at(15)), INV),
    (dict(dz=_at(16)), INV), (dict(dbias=_at(5)), INV), (dict(seqlen=1 << 31), UNS),
])
def test_backward_refusals(libs, kw, expect):
    assert _call(libs[0].jamba_ssm_gated_scan_bwd, _lib.GatedScanBwdParams, BWD, **kw) == expect


def test_sizes(libs):
    L = libs[0]
    assert L.jamba_ssm_gated_scan_ckpt_size(2, 130, 10) == (130 // 64 + 2) * 10 * 4
    assert L.jamba_ssm_gated_scan_ckpt_size(1, 1 << 30, 1 << 20) == ((1 << 24) + 1) << 22
    assert L.jamba_ssm_gated_scan_ckpt_size(-1, 5, 5) == 0
    # every entry that a sequence can address lies inside, however the rows are cut
    for rows in (0, 1, 63, 64, 65, 200):
        for a in range(rows + 1):
            cuts = [0, a, a, rows]
            have = L.jamba_ssm_gated_scan_ckpt_size(3, rows, 1) // 4
            used = [cuts[b] // 64 + b + k for b in range(3)
                    for k in range(-(-(cuts[b + 1] - cuts[b]) // 64))]
            assert len(set(used)) == len(used) and all(v < have for v in used)
    small = L.jamba_ssm_gated_scan_bwd_workspace_size(2, 130, 10, 1)
    assert L.jamba_ssm_gated_scan_bwd_workspace_size(2, 130, 10, 0) > small > 0
    assert L.jamba_ssm_gated_scan_bwd_workspace_size(0, 0, 10, 1) == 0
    assert L.jamba_ssm_gated_scan_bwd_workspace_size(2, -1, 10, 1) == 0


UPD = dict(batch=3, d_inner=50, io_dtype=_lib.BF16, state=_at(1), x=_at(2), g=_at(3), z=_at(4),
           rate=_at(5), bias=_at(6), out=_at(7))


@pytest.mark.parametrize("kw,expect", [
    (dict(struct_size=1), INV), (dict(batch=-1), INV), (dict(d_inner=0), INV),
    (dict(io_dtype=7), INV), (dict(state=None), INV), (dict(x=None), INV), (dict(g=None), INV),
    (dict(out=None), INV), (dict(x_stride=49), INV), (dict(state_indices=_at(8)), INV),
    (dict(out=_at(7) + 1), MIS), (dict(state=_at(1) + 2), MIS), (dict(out=_at(2)), INV),
    (dict(state=_at(3)), INV), (dict(out=_at(1)), INV), (dict(reserved=3), INV),
    (dict(workspace=_at(9), workspace_bytes=0), WSP), (dict(d_inner=(1 << 20) + 1), UNS),
    (dict(state_indices=_at(1), num_slots=5), INV),
])
def test_update_refusals(libs, kw, expect):
    assert _call(libs[0].jamba_ssm_gated_state_update, _lib.GatedStateUpdateParams, UPD,
                 **kw) == expect


QUANT = dict(rows=5, k=100, x_dtype=_lib.F32, x=_at(1), q=_at(2), scale=_at(3))


@pytest.mark.parametrize("kw,expect", [
    (dict(struct_size=3), INV), (dict(rows=-1), INV), (dict(k=0), INV), (dict(x_dtype=2), INV),
    (dict(k=_lib.I8_MAX_K + 1), UNS), (dict(rows=1 << 31), UNS), (dict(x_stride=99), INV),
    (dict(x=None), INV), (dict(q=None), INV), (dict(scale=None), INV), (dict(x=_at(1) + 2), MIS),
    (dict(q=_at(2) + 8), MIS), (dict(scale=_at(3) + 1), MIS), (dict(q=_at(1)), INV),
    (dict(scale=_at(2) + 16), INV), (dict(reserved=1), INV),
])
def test_quant_refusals(libs, kw, expect):
    assert _call(libs[1].jamba_ssm_i8_quant, _lib.I8QuantParams, QUANT, **kw) == expect


PROJ = dict(ntok=5, k=100, n_out=30, out_dtype=_lib.BF16, q=_at(1), q_scale=_at(2), w=_at(3),
            w_scale=_at(4), bias=_at(5), out=_at(6))


@pytest.mark.parametrize("kw,expect", [
    (dict(struct_size=3), INV), (dict(ntok=-1), INV), (dict(k=0), INV), (dict(n_out=0), INV),
    (dict(out_dtype=5), INV), (dict(k=_lib.I8_MAX_K + 1), UNS), (dict(ntok=1 << 31), UNS),
    (dict(n_out=(1 << 24) + 1), UNS), (dict(q=None), INV), (dict(w=None), INV),
    (dict(q_scale=None), INV), (dict(w_scale=None), INV), (dict(out=None), INV),
    (dict(q=_at(1) + 8), MIS), (dict(w=_at(3) + 1), MIS), (dict(bias=_at(5) + 2), MIS),
    (dict(out=_at(6) + 1), MIS), (dict(out=_at(1)), INV), (dict(out=_at(5) + 4), INV),
])
def test_proj_refusals(libs, kw, expect):
    assert _call(libs[1].jamba_ssm_i8_proj, _lib.I8ProjParams, PROJ, **kw) == expect


MAPS = dict(requests=4, max_tokens=50, max_blocks=6, block_size=16, new_lens=_at(1),
            ctx_lens=_at(2), free_blocks=_at(3), num_free_blocks=9, free_slots=_at(4),
            num_free_slots=8, block_tables=_at(5), request_slots=_at(6), cu_seqlens=_at(7),
            positions=_at(8), token_request=_at(9), slot_map=_at(10), state_indices=_at(11),
            initial_indices=_at(12), counts=_at(13))


@pytest.mark.parametrize("kw,expect", [
    (dict(struct_size=3), INV), (dict(requests=-1), INV), (dict(max_tokens=-1), INV),
    (dict(max_blocks=0), INV), (dict(block_size=0), INV), (dict(num_free_blocks=-1), INV),
    (dict(num_free_slots=-1), INV), (dict(requests=(1 << 20) + 1), UNS),
    (dict(max_tokens=(1 << 30) + 1), UNS), (dict(block_size=(1 << 20) + 1), UNS),
    (dict(new_lens=None), INV), (dict(free_blocks=None), INV), (dict(free_slots=None), INV),
    (dict(block_tables=None), INV), (dict(request_slots=None), INV), (dict(cu_seqlens=None), INV),
    (dict(positions=None), INV), (dict(token_request=None), INV), (dict(slot_map=None), INV),
    (dict(state_indices=None), INV), (dict(initial_indices=None), INV), (dict(counts=None), INV),
    (dict(slot_map=_at(10) + 4), MIS), (dict(new_lens=_at(1) + 2), MIS),
    (dict(request_slots=_at(4)), INV), (dict(positions=_at(9)), INV),
    (dict(cu_seqlens=_at(1)), INV), (dict(block_tables=_at(3) + 32), INV),
])
def test_maps_refusals(libs, kw, expect):
    assert _call(libs[1].jamba_ssm_batch_maps, _lib.BatchMapsParams, MAPS, **kw) == expect


def test_valid_calls_without_a_device(libs):
    if _has_gpu():
        pytest.skip("the addresses are not real: only without a GPU")
    L, S = libs
    for fn, cls, base in ((L.jamba_ssm_gated_scan_bwd, _lib.GatedScanBwdParams, BWD),
                          (L.jamba_ssm_gated_state_update, _lib.GatedStateUpdateParams, UPD),
                          (S.jamba_ssm_i8_quant, _lib.I8QuantParams, QUANT),
                          (S.jamba_ssm_i8_proj, _lib.I8ProjParams, PROJ),
                          (S.jamba_ssm_batch_maps, _lib.BatchMapsParams, MAPS)):
        assert _call(fn, cls, base) == _lib.ERR_NO_DEVICE, cls
        assert fn(None, None) == INV
    assert L.jamba_ssm_gated_get_status(None, None) == _lib.ERR_NO_DEVICE
    assert S.jamba_ssm_serve_get_status(None) == _lib.ERR_NO_DEVICE
    # nothing to do needs no pointers
    assert _call(L.jamba_ssm_gated_state_update, _lib.GatedStateUpdateParams, UPD, batch=0,
                 x=None) == _lib.OK
    assert _call(S.jamba_ssm_i8_quant, _lib.I8QuantParams, QUANT, rows=0, x=None) == _lib.OK
    assert _call(S.jamba_ssm_i8_proj, _lib.I8ProjParams, PROJ, ntok=0, q=None) == _lib.OK


def test_python_calls_need_cuda_tensors():
    import torch

    import selective_state_space_26_b200 as jssm
    x, i = torch.zeros(2, 3, 8), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: jssm.jamba_ssm_gated_scan(x, x),
                 lambda: jssm.jamba_ssm_gated_scan_bwd(x, x, x),
                 lambda: jssm.jamba_ssm_gated_state_update(x[0], x[0], x[0]),
                 lambda: jssm.jamba_ssm_i8_quant(x),
                 lambda: jssm.jamba_ssm_i8_proj(x, x, x, x),
                 lambda: jssm.jamba_ssm_batch_maps(i, i[None], i, i, i, max_tokens=2)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()


@pytest.fixture
def two_devices(monkeypatch):
    """The bindings as they are with devices 0 (current) and 1, and a library that
    only writes down which stream it was given while which device was current."""
    import contextlib

    import torch
    now, calls = [0], []

    @contextlib.contextmanager
    def current(dev):
        now.append(torch.device(dev).index)
        yield
        now.pop()

    class Lib:
        def jamba_ssm_gated_get_status(self, ws, stream):
            calls.append((now[-1], ws, stream))
            return 0

        def jamba_ssm_serve_get_status(self, stream):
            calls.append((now[-1], None, stream))
            return 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x100 + (0 | index))
    monkeypatch.setattr(_lib, "gated_lib", Lib)
    monkeypatch.setattr(_lib, "serve_lib", Lib)
    return calls


def test_status_of_a_device_without_an_index(two_devices):
    import torch

    import selective_state_space_26_b200 as jssm
    for status in (jssm.jamba_ssm_gated_get_status, jssm.jamba_ssm_serve_get_status):
        for device in (None, "cuda", torch.device("cuda"), "cuda:0", 0):
            assert status(device=device) == 0
            assert two_devices.pop() == (0, None, 0x100)
        assert status(device="cuda:1") == 0
        assert two_devices.pop() == (1, None, 0x101)


def test_status_of_a_workspace_on_another_device(two_devices, monkeypatch):
    """The stream that is waited for is one of the workspace's device."""
    import torch

    import selective_state_space_26_b200 as jssm
    from selective_state_space_26_b200 import gated

    class Words:
        device = torch.device("cuda:1")
    monkeypatch.setattr(gated, "_workspace", lambda ws, dev: (0x5000, 16))
    assert jssm.jamba_ssm_gated_get_status(workspace=Words()) == 0
    assert two_devices == [(1, 0x5000, 0x101)]


def test_stream_of_another_device_is_refused(two_devices):
    """Before anything is enqueued: the kernel would run there, on this device's
    addresses."""
    from types import SimpleNamespace

    import torch

    import selective_state_space_26_b200 as jssm
    from selective_state_space_26_b200 import _tensors
    there = SimpleNamespace(cuda_stream=0x900, device=torch.device("cuda:1"))
    with pytest.raises(ValueError, match="stream is on cuda:1, expected cuda:0"):
        _tensors.launching(there, torch.device("cuda:0"))
    for status in (jssm.jamba_ssm_gated_get_status, jssm.jamba_ssm_serve_get_status):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            status(stream=there, device=0)
    assert two_devices == []
