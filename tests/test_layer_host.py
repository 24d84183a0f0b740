"""include/layer.h on the host: exports, struct layout, and the refusal of every
invalid call before anything reaches the GPU (addresses are fake and never
dereferenced; each call fails validation or has no work); and properties of the
generated gfx950 code."""
import ctypes
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

import selective_state_update_ssu_amd as ssu
from selective_state_update_ssu_amd import _abi, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "layer.h")
INV, UNS = _abi.SSU_ERR_INVALID_ARGUMENT, _abi.SSU_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssu.library_path()):
        build.build()
    return ssu.library()


def addr(i):
    return 0x7F0000000000 + i * (1 << 34)


def test_exports_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^(?:int|size_t)\s+(ssu_\w+)\s*\(", text, re.M)
    assert sorted(names) == sorted(_abi.LAYER_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layout_matches_header(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "layer.h"', "int main(void){"]
    want = {}
    for cname, cls in (("ssu_conv_args", _abi.ConvArgs), ("ssu_scan_args", _abi.ScanArgs),
                       ("ssu_cache_block", _abi.CacheBlock), ("ssu_cache_args", _abi.CacheArgs)):
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        want[cname] = ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            lines.append(f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));')
            want[f"{cname}.{f}"] = getattr(cls, f).offset
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{os.path.dirname(HEADER)}", str(src),
                    "-o", str(exe)], check=True)
    text = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert {k: int(v) for k, v in (l.split() for l in text.splitlines())} == want


def call(lib, entry, args, kw):
    for k, v in kw.items():
        assert hasattr(args, k), k
        setattr(args, k, v)
    return getattr(lib, entry)(ctypes.byref(args), None), lib.ssu_last_error().decode()


def conv(lib, varlen=True, **kw):
    a = _abi.ConvArgs(
        struct_size=ctypes.sizeof(_abi.ConvArgs), io_dtype=_abi.SSU_BF16, conv_state=addr(1),
        nslots=8, slot_stride=3 * 64, x=addr(2), x_stride=128, out=addr(3), out_stride=64,
        weight=addr(4), bias=addr(5), rows=10, dim=64, width=4, silu=1,
        cu_seqlens=addr(6) if varlen else None, nseq=3 if varlen else 10,
        has_initial=addr(7) if varlen else None, slots=addr(8), pad_slot_id=-1)
    return call(lib, "ssu_conv1d_varlen" if varlen else "ssu_conv1d_update", a, kw)


@pytest.mark.parametrize("varlen,kw,code,needle", [
    (True, dict(struct_size=8), INV, "struct_size"),
    (True, dict(io_dtype=3), INV, "io_dtype"),
    (True, dict(rows=-1), INV, "sizes"),
    (True, dict(dim=0), INV, "sizes"),
    (True, dict(nslots=0), INV, "sizes"),
    (True, dict(nseq=-1), INV, "sizes"),
    (True, dict(width=5), UNS, "width 5"),
    (True, dict(width=1), UNS, "width 1"),
    (True, dict(x_stride=-1), INV, "x_stride"),
    (True, dict(out_stride=63), INV, "out_stride"),
    (True, dict(slot_stride=191), INV, "slot_stride"),
    (True, dict(cu_dtype=2), INV, "cu_dtype"),
    (True, dict(slot_dtype=2), INV, "slot_dtype"),
    (True, dict(cu_seqlens=None), INV, "cu_seqlens"),
    (True, dict(x=None), INV, "x must not"),
    (True, dict(out=None), INV, "out must not"),
    (True, dict(weight=None), INV, "weight must not"),
    (True, dict(conv_state=None), INV, "conv_state must not"),
    (True, dict(x=addr(2) + 1), INV, "aligned"),
    (True, dict(out=addr(2) + 64), INV, "out overlaps x"),
    (True, dict(out=addr(1)), INV, "out overlaps conv_state"),
    (True, dict(conv_state=addr(5)), INV, "conv_state overlaps bias"),
    (True, dict(rows=1 << 40, x_stride=0, out=1 << 48), UNS, "too many rows"),
    (False, dict(cu_seqlens=addr(6)), INV, "belong to"),
    (False, dict(has_initial=addr(6)), INV, "belong to"),
    (False, dict(nseq=9), INV, "nseq"),
])
def test_conv_rejects(lib, varlen, kw, code, needle):
    rc, msg = conv(lib, varlen, **kw)
    assert rc == code, (rc, msg)
    assert needle in msg, msg


def scan(lib, varlen=True, **kw):
    a = _abi.ScanArgs(
        struct_size=ctypes.sizeof(_abi.ScanArgs), state_dtype=_abi.SSU_F32, state=addr(1), nslots=8,
        slot_stride=64 * 16, rows=10, dim=64, dstate=16, ngroups=2, x=addr(2), z=addr(3),
        dt=addr(4), B=addr(5), C=addr(6), out=addr(7), x_stride=64, z_stride=128, dt_stride=64,
        B_stride=40, C_stride=40, out_stride=64, io_dtype=_abi.SSU_BF16, dt_dtype=_abi.SSU_F32,
        A=addr(8), D=addr(9), dt_bias=addr(10), dt_softplus=1,
        cu_seqlens=addr(11) if varlen else None, nseq=3 if varlen else 10,
        has_initial=addr(12) if varlen else None, slots=addr(13), pad_slot_id=-1,
        workspace=addr(14) if varlen else None, workspace_bytes=(1 << 26) if varlen else 0)
    return call(lib, "ssu_scan_varlen" if varlen else "ssu_scan_update", a, kw)


@pytest.mark.parametrize("varlen,kw,code,needle", [
    (True, dict(struct_size=8), INV, "struct_size"),
    (True, dict(reserved=1), INV, "reserved"),
    (True, dict(state_dtype=9), INV, "state_dtype"),
    (True, dict(io_dtype=-1), INV, "io_dtype"),
    (True, dict(dt_dtype=_abi.SSU_F16), INV, "dt must"),
    (True, dict(rows=-1), INV, "sizes"),
    (True, dict(ngroups=0), INV, "sizes"),
    (True, dict(ngroups=3), INV, "multiple of ngroups"),
    (True, dict(dstate=24), UNS, "dstate 24"),
    (True, dict(dstate=512), UNS, "dstate 512"),
    (True, dict(rows=1 << 31), UNS, "below 2^31"),
    (True, dict(dim=1 << 30), UNS, "below 2^31"),
    (True, dict(slot_stride=1023), INV, "slot_stride"),
    (True, dict(B_stride=-1), INV, "strides"),
    (True, dict(out_stride=60), INV, "out_stride"),
    (True, dict(cu_dtype=4), INV, "cu_dtype"),
    (True, dict(slot_dtype=4), INV, "slot_dtype"),
    (True, dict(state=None), INV, "state must not"),
    (True, dict(out=None), INV, "out must not"),
    (True, dict(dt=None), INV, "dt must not"),
    (True, dict(A=None), INV, "A must not"),
    (True, dict(cu_seqlens=None), INV, "cu_seqlens must not"),
    (True, dict(B=addr(5) + 1), INV, "B must be aligned"),
    (True, dict(dt=addr(4) + 2), INV, "dt must be aligned"),
    (True, dict(out=addr(7) + 1), INV, "out must be aligned"),
    (True, dict(state=addr(1) + 8), UNS, "16-byte aligned"),
    (True, dict(slot_stride=1026), UNS, "16-byte aligned"),
    (True, dict(rows=4096, workspace=None), INV, "workspace"),
    (True, dict(rows=4096, workspace=addr(14) + 16), INV, "workspace"),
    (True, dict(rows=4096, workspace_bytes=100), INV, "workspace"),
    (True, dict(rows=4096, workspace=addr(2)), INV, "workspace overlaps x"),
    (True, dict(out=addr(2)), INV, "out overlaps x"),
    (True, dict(state=addr(8)), INV, "state overlaps A"),
    (True, dict(state=addr(7)), INV, "state overlaps out"),
    (False, dict(workspace=addr(14)), INV, "belong to"),
    (False, dict(cu_seqlens=addr(11)), INV, "belong to"),
    (False, dict(nseq=4), INV, "nseq"),
])
def test_scan_rejects(lib, varlen, kw, code, needle):
    rc, msg = scan(lib, varlen, **kw)
    assert rc == code, (rc, msg)
    assert needle in msg, msg


def test_scan_workspace_covers_a_cut_of_every_sequence(lib):
    """Scratch grows with every size, and refuses nonsense with 0."""
    base = (1000, 3, 64, 16, 2)
    size = lib.ssu_scan_workspace_bytes(*base)
    assert size >= 1000 // 64 * 64 * 16 * 4
    for i in range(5):
        more = list(base)
        more[i] *= 8
        assert lib.ssu_scan_workspace_bytes(*more) >= size, i
    assert lib.ssu_scan_workspace_bytes(-1, 3, 64, 16, 2) == 0
    assert lib.ssu_scan_workspace_bytes(10, 3, 0, 16, 2) == 0


def cache(lib, entry, blocks=((addr(20), 64, 64),), **kw):
    arr = (_abi.CacheBlock * max(1, len(blocks)))(*[_abi.CacheBlock(*b) for b in blocks])
    a = _abi.CacheArgs(struct_size=ctypes.sizeof(_abi.CacheArgs), delta=-1, refcount=addr(1),
                       nslots=16, caches=arr, ncaches=len(blocks), src=addr(2), dst=addr(3), n=4,
                       ids=addr(4), remap=addr(5), plan=addr(6))
    return call(lib, entry, a, kw)


@pytest.mark.parametrize("entry,kw,needle", [
    ("ssu_cache_alloc", dict(struct_size=1), "struct_size"),
    ("ssu_cache_alloc", dict(nslots=-1), "nslots"),
    ("ssu_cache_alloc", dict(nslots=1 << 31), "nslots"),
    ("ssu_cache_alloc", dict(n=-1), "n must"),
    ("ssu_cache_alloc", dict(refcount=None), "refcount"),
    ("ssu_cache_alloc", dict(refcount=addr(1) + 2), "aligned"),
    ("ssu_cache_alloc", dict(ids=None), "ids"),
    ("ssu_cache_adjust", dict(delta=2), "delta"),
    ("ssu_cache_adjust", dict(src=None), "src"),
    ("ssu_cache_adjust", dict(src_dtype=3), "src_dtype"),
    ("ssu_cache_adjust", dict(src=addr(2) + 4, src_dtype=_abi.SSU_I64), "aligned"),
    ("ssu_cache_copy", dict(dst=None), "dst"),
    ("ssu_cache_copy", dict(dst_dtype=-1), "dst_dtype"),
    ("ssu_cache_copy", dict(ncaches=-1), "ncaches"),
    ("ssu_cache_copy", dict(blocks=((None, 64, 64),)), "base"),
    ("ssu_cache_copy", dict(blocks=((addr(20), 64, 32),)), "stride_bytes"),
    ("ssu_cache_copy", dict(blocks=((addr(20), -1, 32),)), "slot_bytes"),
    ("ssu_cache_compact", dict(remap=None), "remap"),
    ("ssu_cache_compact", dict(plan=None), "plan"),
    ("ssu_cache_compact", dict(refcount=None), "refcount"),
    ("ssu_cache_compact", dict(blocks=((addr(20), 64, 63),)), "stride_bytes"),
])
def test_cache_rejects(lib, entry, kw, needle):
    rc, msg = cache(lib, entry, **kw)
    assert rc == INV, (rc, msg)
    assert needle in msg, msg


def test_no_work_is_ok(lib):
    for varlen in (True, False):
        zero = dict(rows=0, nseq=0, x=None, out=None)
        assert conv(lib, varlen, **zero) == (_abi.SSU_OK, "")
        assert scan(lib, varlen, **zero) == (_abi.SSU_OK, "")
    assert conv(lib, True, nseq=0)[0] == _abi.SSU_OK
    assert scan(lib, True, nseq=0)[0] == _abi.SSU_OK
    assert cache(lib, "ssu_cache_alloc", n=0, ids=None)[0] == _abi.SSU_OK
    assert cache(lib, "ssu_cache_adjust", n=0, src=None)[0] == _abi.SSU_OK
    assert cache(lib, "ssu_cache_copy", n=0, src=None)[0] == _abi.SSU_OK
    assert cache(lib, "ssu_cache_copy", blocks=())[0] == _abi.SSU_OK
    assert cache(lib, "ssu_cache_compact", nslots=0, refcount=None)[0] == _abi.SSU_OK


def test_null_args(lib):
    for entry in _abi.LAYER_EXPORTS:
        if entry != "ssu_scan_workspace_bytes":
            assert getattr(lib, entry)(None, None) == INV, entry


def test_binding_refuses_host_tensors():
    import torch
    x, w = torch.zeros(2, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="GPU"):
        ssu.causal_conv1d_update(torch.zeros(2, 3, 8), x, w)
    with pytest.raises(ValueError, match="GPU"):
        ssu.selective_scan_update(torch.zeros(2, 8, 16), x, x, torch.zeros(8, 16),
                                  torch.zeros(2, 1, 16), torch.zeros(2, 1, 16))
    with pytest.raises(ValueError, match="GPU"):
        ssu.cache_alloc(torch.zeros(4, dtype=torch.int32), 1)
    with pytest.raises(ValueError, match="GPU"):
        ssu.cache_copy([torch.zeros(4, 3)], torch.zeros(1, dtype=torch.int32),
                       torch.zeros(1, dtype=torch.int32))


# ------------------------------------------------------------------ generated code

UNITS = ["layer_conv.hip", "layer_scan_f32.hip", "layer_scan_f16.hip", "layer_scan_bf16.hip",
         "layer_cache.hip"]


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    out = tmp_path_factory.mktemp("layer_isa")

    def one(unit):
        path = os.path.join(str(out), unit + ".s")
        flags = [f for f in build.CXXFLAGS if f != "-fPIC"]
        r = subprocess.run([build.HIPCC, *flags, "--cuda-device-only", "-S",
                            os.path.join(build.CSRC, unit), "-o", path],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return unit, open(path).read()

    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    with ThreadPoolExecutor(len(UNITS)) as ex:
        return dict(ex.map(one, UNITS))


def test_no_scratch_no_spills_no_packed_fp32(asm):
    for unit, text in asm.items():
        assert not re.search(r"v_pk_(fma|mul|add)_f32", text), unit
        for field in ("private_segment_fixed_size", "vgpr_spill_count"):
            values = re.findall(rf"\.{field}:\s*(\d+)", text)
            assert values and set(values) == {"0"}, (unit, field)


def test_scan_keeps_its_exponentials_to_the_decays(asm):
    """Every scan instance uses the hardware's exponential and passes what its waves share
    through LDS, with one barrier per tile."""
    for unit, want in (("layer_scan_f32.hip", 18), ("layer_scan_f16.hip", 36),
                       ("layer_scan_bf16.hip", 36)):
        bodies = [(m.group(1), asm[unit][m.end():asm[unit].find(".Lfunc_end", m.end())])
                  for m in re.finditer(r"^(_Z\w*scan_kernel\w+):", asm[unit], re.M)]
        assert len(bodies) == want, (unit, len(bodies))
        for name, body in bodies:
            assert "v_exp_f32" in body and "ds_read" in body, name
            # One before the loop, one in each of its two copies of a tile's body, and one
            # for the sums of a first pass.
            assert len(re.findall(r"\ts_barrier", body)) <= 4, name


def test_scan_scratch_is_the_calls_own():
    """The scan's passes hand each other states through its scratch: it takes no part in the
    prefill's buffers, which calls of a stream share and a larger call replaces."""
    from selective_state_update_ssu_amd import layer
    binding = layer._load()
    assert not hasattr(layer, "_cached_workspace")
    for n in (15, 17):
        with pytest.raises(TypeError, match="number of arguments"):
            binding.scan(*[None] * n)
    with pytest.raises(ValueError, match="state must be a tensor"):
        binding.scan(*[None] * 16)


def test_binding_switches_to_the_tensors_gpu():
    """The native binding holds a device guard over its launches (what it does with two GPUs is
    a test of its own, which needs them)."""
    from selective_state_update_ssu_amd import layer
    layer._load()
    names = subprocess.run(["nm", "-D", "--undefined-only", layer.binding_path()],
                           capture_output=True, text=True, check=True).stdout
    assert "device_guard_impl_registry" in names


def test_scan_of_16_elements_per_lane_keeps_its_waves(asm):
    """States of 64 and 128 (16 elements per lane) with 16-bit io: four waves per SIMD take 128
    registers each."""
    for unit in ("layer_scan_f16.hip", "layer_scan_bf16.hip"):
        found = re.findall(r"\.name:\s+_ZN5layer11scan_kernelI\S*?Li(64|128)ELi\d\S*"
                           r".*?\.vgpr_count:\s+(\d+)", asm[unit], re.S)
        assert len(found) == 12, unit
        assert all(int(n) <= 128 for _, n in found), (unit, found)


def test_columns_of_one_buffer_do_not_overlap(lib):
    """Operands in disjoint columns of rows of one buffer pass the overlap checks (the calls end at
    a later refusal: too many rows or workgroups for one launch), touching ones do not."""
    far = 1 << 56
    many = dict(rows=1 << 40, x=far, x_stride=128, out_stride=128)
    for out in (far + 128, far - 128, far + 256 * 7 + 128):
        rc, msg = conv(lib, out=out, **many)
        assert rc == UNS and "too many rows" in msg, (out - far, msg)
    for out in (far + 126, far + 130, far, far - 126, far + 256 * 7):
        rc, msg = conv(lib, out=out, **many)
        assert rc == INV and "out overlaps x" in msg, (out - far, msg)
    rc, msg = conv(lib, out=far + 128, **dict(many, x_stride=64))
    assert rc == INV and "out overlaps x" in msg, msg

    wide = dict(nseq=1 << 30, x_stride=256, out_stride=256, B_stride=256)
    for kw in (dict(out=addr(2) + 128), dict(out=addr(2) + 192, B=addr(2) + 128),
               dict(out=addr(2) - 192)):
        rc, msg = scan(lib, **wide, **kw)
        assert rc == _abi.SSU_ERR_LAUNCH and "launch failed" in msg, (kw, msg)
    for kw, needle in ((dict(out=addr(2) + 126), "out overlaps x"),
                       (dict(out=addr(2) + 192, B=addr(2) + 130), "out overlaps B"),
                       (dict(out=addr(2) + 386), "out overlaps x")):
        rc, msg = scan(lib, **wide, **kw)
        assert rc == INV and needle in msg, (kw, msg)


@pytest.mark.parametrize("torch_there", [False, True])
def test_build_of_the_library_does_not_need_the_binding(torch_there, monkeypatch, tmp_path):
    """Without torch, or where the binding does not compile, the C library is still built."""
    import sys
    ran, moved = [], []

    def run(cmd):
        ran.append(cmd)
        if any(c.endswith(build.BINDING_SOURCE) for c in cmd):
            raise RuntimeError("the binding does not compile")
        return ""

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build.os, "replace", lambda a, b: moved.append(b))
    if torch_there:
        monkeypatch.setattr(build, "_binding_flags", lambda: [])
        with pytest.raises(RuntimeError, match="does not compile"):
            build.build()
    else:
        monkeypatch.setitem(sys.modules, "torch", None)
        assert build.build() == build.LIBRARY
    assert moved == [build.LIBRARY, build.STREAM_LIBRARY]
    assert sum("-shared" in cmd for cmd in ran) == 2


def test_binding_refuses_a_tensor_for_a_list_of_caches():
    """A tensor is a sequence of its slots: taken as caches they would be copied inside."""
    import torch
    ids = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="list of tensors"):
        ssu.cache_copy(torch.zeros(4, 4, 3), ids, ids)
