"""The C ABI on the host: the library loads, exports what include/*.h declare,
agrees with the ctypes mirror on struct layout, and rejects every invalid call
before touching the GPU. No call here reaches a kernel launch: each one either
fails validation or has no work, so these run on machines without a GPU."""
import ctypes
import os
import re
import subprocess

import pytest

from selective_state_update_ssu_amd import _abi
import selective_state_update_ssu_amd as ssu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssu.h")
HEADERS = [HEADER, os.path.join(ROOT, "include", "ssd.h")]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssu.library_path()):
        from selective_state_update_ssu_amd import build
        build.build()
    return ssu.library()


def declared_functions():
    names = set()
    for h in HEADERS:
        text = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        names |= set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(ssu_\w+)\s*\(", text, re.M))
    return sorted(names)


def test_exports_every_declared_function(lib):
    names = declared_functions()
    assert names == sorted(_abi.EXPORTS), names
    for n in names:
        assert hasattr(lib, n), n
    nm = subprocess.run(["nm", "-D", "--defined-only", ssu.library_path()],
                        capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r" T (\w+)$", nm, re.M))
    assert set(names) <= exported


def test_version(lib):
    assert lib.ssu_version() == _abi.ABI_VERSION


def test_struct_layout_matches_header(tmp_path):
    """Offsets and sizes of every field, as the C compiler lays them out."""
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "ssu.h"', '#include "ssd.h"',
             "int main(void){"]
    checks = []
    for cname, cls in (("ssu_operands", _abi.Operands), ("ssu_one_token_args", _abi.OneTokenArgs),
                       ("ssu_packed_args", _abi.PackedArgs), ("ssu_ring_args", _abi.RingArgs),
                       ("ssu_ssd_args", _abi.SsdArgs)):
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        checks.append((cname, ctypes.sizeof(cls)))
        for fname, _ in cls._fields_:
            lines.append(f'printf("{cname}.{fname} %zu\\n", offsetof({cname}, {fname}));')
            checks.append((f"{cname}.{fname}", getattr(cls, fname).offset))
    lines.append("return 0;}")
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", f"-I{os.path.dirname(HEADER)}", str(src), "-o", str(exe)],
                   check=True)
    got = dict(l.rsplit(" ", 1) for l in subprocess.run([str(exe)], capture_output=True,
                                                         text=True, check=True).stdout.split("\n") if l)
    for key, want in checks:
        assert int(got[key]) == want, (key, got[key], want)


# Fake, never-dereferenced device addresses, 256-byte aligned and far apart.
def addr(i):
    return 0x7F0000000000 + i * (1 << 32)


def good_operands(**kw):
    op = _abi.Operands(
        state=addr(1), state_dtype=_abi.SSU_F32, nslots=8, nheads=8, headdim=64, dstate=128,
        ngroups=2, x=addr(2), B=addr(3), C=addr(4), z=addr(5), out=addr(6),
        io_dtype=_abi.SSU_BF16, dt=addr(7), dt_per_dim=0, A=addr(8), D=addr(9),
        dt_bias=addr(10), dt_softplus=1, pad_slot_id=-1, disable_state_update=0,
        heads_per_block=0, loads_per_lane=0, tile_order=0)
    for k, v in kw.items():
        setattr(op, k, v)
    return op


def one_token(lib, batch=4, **kw):
    a = _abi.OneTokenArgs(struct_size=ctypes.sizeof(_abi.OneTokenArgs), op=good_operands(),
                          batch=batch, src_slots=addr(11), src_dtype=_abi.SSU_I32,
                          dst_slots=None, dst_dtype=0)
    for k, v in kw.items():
        if hasattr(a.op, k) and k not in ("struct_size",):
            setattr(a.op, k, v)
        else:
            setattr(a, k, v)
    rc = lib.ssu_one_token(ctypes.byref(a), None)
    return rc, lib.ssu_last_error().decode()


def packed(lib, **kw):
    a = _abi.PackedArgs(struct_size=ctypes.sizeof(_abi.PackedArgs), op=good_operands(),
                        rows=10, nseq=4, cu_seqlens=addr(12), num_accepted=addr(13),
                        meta_dtype=_abi.SSU_I32, src_table=addr(14), src_dtype=_abi.SSU_I32,
                        src_seq_stride=4, src_step_stride=1, dst_table=addr(15),
                        dst_dtype=_abi.SSU_I32, dst_seq_stride=4, dst_step_stride=1, steps=4)
    for k, v in kw.items():
        if hasattr(a.op, k):
            setattr(a.op, k, v)
        else:
            setattr(a, k, v)
    rc = lib.ssu_packed_varlen(ctypes.byref(a), None)
    return rc, lib.ssu_last_error().decode()


INV, UNS = _abi.SSU_ERR_INVALID_ARGUMENT, _abi.SSU_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code,needle", [
    (dict(ngroups=0), INV, "positive"),
    (dict(ngroups=3), INV, "multiple of ngroups"),
    (dict(nslots=0), INV, "positive"),
    (dict(dstate=48), UNS, "dstate 48"),
    (dict(state_dtype=7), INV, "state_dtype"),
    (dict(io_dtype=-1), INV, "io_dtype"),
    (dict(dt_per_dim=2), INV, "dt_per_dim"),
    (dict(heads_per_block=3), INV, "heads_per_block"),
    (dict(heads_per_block=8), INV, "heads_per_block"),
    (dict(loads_per_lane=3), INV, "loads_per_lane"),
    (dict(loads_per_lane=8), INV, "loads_per_lane"),
    (dict(tile_order=4), INV, "tile_order"),
    (dict(nheads=12, ngroups=4, heads_per_block=2), INV, "divide"),
    (dict(dstate=256, heads_per_block=4), UNS, "exceeds"),
    (dict(state=0), INV, "state must not be NULL"),
    (dict(x=0), INV, "x must not be NULL"),
    (dict(A=0), INV, "A must not be NULL"),
    (dict(out=0), INV, "out must not be NULL"),
    (dict(state=addr(1) + 8), UNS, "16-byte aligned"),
    (dict(x=addr(2) + 1), INV, "aligned"),
    (dict(out=addr(2) + 64), INV, "out overlaps x"),
    (dict(out=addr(1) + 4096), INV, "out overlaps state"),
    (dict(batch=-1), INV, "batch"),
    (dict(src_dtype=5), INV, "src_dtype"),
    (dict(struct_size=8), INV, "struct_size"),
])
def test_one_token_rejects(lib, kw, code, needle):
    rc, msg = one_token(lib, **kw)
    assert rc == code, (rc, msg)
    assert needle in msg, msg


def test_one_token_empty_batch_is_ok(lib):
    rc, msg = one_token(lib, batch=0)
    assert rc == _abi.SSU_OK and msg == ""


def test_null_args(lib):
    assert lib.ssu_one_token(None, None) == INV
    assert lib.ssu_packed_varlen(None, None) == INV


@pytest.mark.parametrize("kw,code,needle", [
    (dict(src_table=None), INV, "src_table is required"),
    (dict(cu_seqlens=None), INV, "cu_seqlens must not be NULL"),
    (dict(seq_len=2), INV, "either cu_seqlens or seq_len"),
    (dict(cu_seqlens=None, seq_len=3), INV, "nseq * seq_len"),
    (dict(seq_len=-1), INV, "seq_len"),
    (dict(meta_dtype=3), INV, "meta_dtype"),
    (dict(steps=0), INV, "steps"),
    (dict(src_seq_stride=-1), INV, "strides"),
    (dict(dst_step_stride=-2), INV, "strides"),
    (dict(rows=-1), INV, "rows"),
    (dict(dst_dtype=9), INV, "dst_dtype"),
    (dict(dstate=100), UNS, "dstate 100"),
    (dict(heads_per_block=4), UNS, "exceeds"),
    (dict(struct_size=4), INV, "struct_size"),
])
def test_packed_rejects(lib, kw, code, needle):
    rc, msg = packed(lib, **kw)
    assert rc == code, (rc, msg)
    assert needle in msg, msg


def test_packed_without_work_is_ok(lib):
    assert packed(lib, nseq=0)[0] == _abi.SSU_OK
    assert packed(lib, rows=0)[0] == _abi.SSU_OK


def ring(lib, commit=False, **kw):
    a = _abi.RingArgs(struct_size=ctypes.sizeof(_abi.RingArgs), ring_start=addr(20),
                      prev_num_accepted=addr(21), prev_query_len=addr(22),
                      tracker_dtype=_abi.SSU_I32, num_states=64, slots=addr(23),
                      slot_dtype=_abi.SSU_I32, slot_stride=1, n=8, num_accepted=addr(24),
                      query_start_loc=addr(25), meta_dtype=_abi.SSU_I32, reset=0,
                      logical_window=4, ring_buffer_len=16, pad_slot_id=-1)
    for k, v in kw.items():
        setattr(a, k, v)
    f = lib.ssu_ring_commit if commit else lib.ssu_ring_update
    return f(ctypes.byref(a), None), lib.ssu_last_error().decode()


@pytest.mark.parametrize("commit,kw,needle", [
    (False, dict(struct_size=3), "struct_size"),
    (False, dict(n=-1), "n and num_states"),
    (False, dict(slot_stride=-1), "slot_stride"),
    (False, dict(tracker_dtype=2), "tracker_dtype"),
    (False, dict(slot_dtype=7), "slot_dtype"),
    (False, dict(ring_buffer_len=0), "ring_buffer_len"),
    (False, dict(logical_window=-1), "logical_window"),
    (False, dict(slots=None), "slots"),
    (False, dict(prev_query_len=None), "tracker pointers"),
    (False, dict(ring_start=addr(20) + 2), "aligned"),
    (True, dict(meta_dtype=5), "meta_dtype"),
    (True, dict(query_start_loc=None), "query_start_loc"),
    (True, dict(ring_buffer_len=-3), "ring_buffer_len"),
])
def test_ring_rejects(lib, commit, kw, needle):
    rc, msg = ring(lib, commit, **kw)
    assert rc == INV, (rc, msg)
    assert needle in msg, msg


def test_ring_reset_needs_no_ring_length_and_empty_is_ok(lib):
    assert ring(lib, n=0)[0] == _abi.SSU_OK
    assert ring(lib, True, n=0)[0] == _abi.SSU_OK
    # reset ignores the window parameters, but still checks its pointers
    assert ring(lib, reset=1, ring_buffer_len=0, slots=None)[0] == INV


def test_binding_refuses_host_tensors():
    """No CPU fallback: host tensors are rejected before any launch."""
    import torch
    from selective_state_update_ssu_amd import workloads as wl
    w = wl.tiny("cpu")
    with pytest.raises(ValueError, match="GPU"):
        ssu.ssu_one_token(w.state, w.x, w.dt, w.A, w.B, w.C, D=w.D, dt_bias=w.dt_bias)


def test_product_never_touches_the_oracle():
    pkg = os.path.join(ROOT, "selective_state_update_ssu_amd")
    for dirpath, _, files in os.walk(pkg):
        for f in files:
            if f.endswith((".py", ".hip", ".hpp", ".h", ".cpp")):
                text = open(os.path.join(dirpath, f)).read()
                assert "oracle" not in text.lower(), os.path.join(dirpath, f)


# ------------------------------------------------------------------ SSD prefill

def ssd(lib, **kw):
    a = _abi.SsdArgs(
        struct_size=ctypes.sizeof(_abi.SsdArgs), tokens=1000, nheads=8, headdim=64, dstate=128,
        ngroups=2, chunk_size=256, nchunks=6, batch=3, x=addr(1), dt=addr(2), A=addr(3),
        B=addr(4), C=addr(5), D=addr(6), z=addr(7), dt_bias=addr(8), io_dtype=_abi.SSU_BF16,
        dt_dtype=_abi.SSU_F32, D_per_dim=0, dt_softplus=1, dt_min=0.0, dt_max=float("inf"),
        cu_chunk_seqlens=addr(9), seq_idx=addr(10), last_chunk_indices=addr(11),
        meta_dtype=_abi.SSU_I32, state_dtype=_abi.SSU_F32, initial_states=addr(12),
        out=addr(13), states=addr(14), return_intermediate_states=0, reserved=0,
        workspace=addr(15), workspace_bytes=1 << 30)
    for k, v in kw.items():
        setattr(a, k, v)
    rc = lib.ssu_ssd_prefill(ctypes.byref(a), None)
    return rc, lib.ssu_last_error().decode()


@pytest.mark.parametrize("kw,code,needle", [
    (dict(struct_size=8), INV, "struct_size"),
    (dict(ngroups=3), INV, "divisible"),
    (dict(nheads=0), INV, "positive"),
    (dict(chunk_size=0), INV, "chunk_size"),
    (dict(nchunks=0), INV, "two entries"),
    (dict(io_dtype=_abi.SSU_F32), INV, "fp16/bf16"),
    (dict(dt_dtype=9), INV, "dt must be"),
    (dict(state_dtype=9), INV, "state_dtype"),
    (dict(meta_dtype=4), INV, "int32 or int64"),
    (dict(dt_min=1.0, dt_max=0.5), INV, "dt_limit"),
    (dict(x=0), INV, "required"),
    (dict(A=0), INV, "A is required"),
    (dict(seq_idx=0), INV, "required"),
    (dict(last_chunk_indices=0), INV, "last_chunk_indices"),
    (dict(states=0), INV, "states is required"),
    (dict(headdim=80), UNS, "no kernel"),
    (dict(dstate=512), UNS, "no kernel"),
    (dict(headdim=320), UNS, "no kernel"),
    (dict(chunk_size=64), UNS, "no kernel"),
    (dict(x=addr(1) + 8), UNS, "16-byte aligned"),
    (dict(states=addr(14) + 4), UNS, "states must be 16-byte aligned"),
    (dict(workspace_bytes=1024), INV, "workspace"),
    (dict(workspace=addr(15) + 16), INV, "workspace"),
    (dict(out=addr(1) + 64), INV, "out overlaps x"),
    (dict(states=addr(12) + 64), INV, "states overlaps initial_states"),
    (dict(reserved=1), INV, "reserved"),
])
def test_ssd_rejects(lib, kw, code, needle):
    rc, msg = ssd(lib, **kw)
    assert rc == code, (rc, msg)
    assert needle in msg, msg


def test_ssd_workspace_bytes(lib):
    n = lib.ssu_ssd_workspace_bytes(6, 3, 8, 64, 128, 2, 256)
    # entering states (io-type high parts and low bytes: three bytes per
    # element), C B^T per chunk and group (fp32), decay exponents, the request
    # list, chunk descriptors (16 bytes), chunk-state weights (fp32), the scan's
    # steps and running sums (two fp32 per token and head), the runs.
    need = (6 * 8 * 64 * 128 * 3 + 6 * 2 * 256 * 256 * 4 + 6 * 8 * 4 + 6 * 4 + 3 * 4 + 6 * 16
            + 6 * 8 * 256 * 4 + 6 * 8 * 256 * 8 + 3 * 6 * 4 + 4)
    assert need <= n <= need + 12 * 256 and n % 256 == 0
    assert lib.ssu_ssd_workspace_bytes(-1, 3, 8, 64, 128, 2, 256) == 0


def test_error_text_is_per_thread(lib):
    """Two host threads fail with different messages at the same time; each
    reads back its own, and a later successful (empty) call clears only the
    caller's text."""
    import threading

    both_failed = threading.Barrier(2)
    a_cleared = threading.Event()
    seen = {}

    def worker(name, kw):
        rc, _ = one_token(lib, **kw)
        both_failed.wait()
        seen[name, "rc"] = rc
        seen[name, "after both"] = lib.ssu_last_error().decode()
        if name == "a":
            seen["a", "empty rc"], seen["a", "after empty"] = one_token(lib, batch=0)
            a_cleared.set()
        else:
            a_cleared.wait()
            seen["b", "after a cleared"] = lib.ssu_last_error().decode()

    threads = [threading.Thread(target=worker, args=("a", dict(ngroups=3))),
               threading.Thread(target=worker, args=("b", dict(dstate=48)))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=30)
    assert seen["a", "rc"] == INV and "multiple of ngroups" in seen["a", "after both"]
    assert seen["b", "rc"] == UNS and "dstate 48" in seen["b", "after both"]
    assert seen["a", "empty rc"] == _abi.SSU_OK and seen["a", "after empty"] == ""
    assert "dstate 48" in seen["b", "after a cleared"]


def test_per_head_views_host():
    """The binding's per-head parameter forms (pure host logic, CPU tensors):
    tied views with size 1 or stride 0 after the head dimension give the
    per-head vector; a parameter that varies along dim or dstate is refused."""
    import torch
    from selective_state_update_ssu_amd import _per_head

    H, P, N = 4, 8, 16
    v = torch.arange(H, dtype=torch.float32) - 1.5
    for form in (v, v[:, None], v[:, None].expand(H, P), v[:, None, None].expand(H, P, N),
                 v[:, None, None].expand(H, 1, N), v[:, None, None].contiguous()):
        got = _per_head("D", form, H, P, N)
        assert got.shape == (H,) and torch.equal(got, v), tuple(form.shape)
    with pytest.raises(NotImplementedError):
        _per_head("D", torch.randn(H, P), H, P, N)            # per channel
    with pytest.raises(NotImplementedError):
        _per_head("A", torch.randn(H, P, 1).expand(H, P, N), H, P, N)  # varies along dim
    with pytest.raises(ValueError):
        _per_head("D", v[:, None].expand(H, P + 1), H, P, N)  # wrong dim size
    with pytest.raises(NotImplementedError):
        _per_head("D", v.double(), H, P, N)


def test_ssd_workspace_api_host(lib):
    """The prefill's workspace figure for callers that bring their own buffer,
    and the cache reset (nothing cached on a machine that ran no prefill)."""
    n = lib.ssu_ssd_workspace_bytes(6, 3, 8, 64, 128, 2, 256)
    assert ssu.ssd_workspace_bytes(6, 3, 8, 64, 128, 2, 256) == n + 255
    ssu.reset_ssd_workspaces()
    assert ssu._ssd_workspaces == {}


def _ssd_args(**kw):
    a = _abi.SsdArgs()
    a.struct_size = ctypes.sizeof(_abi.SsdArgs)
    a.tokens, a.nheads, a.headdim, a.dstate, a.ngroups = 300, 4, 64, 128, 2
    a.chunk_size, a.nchunks, a.batch = 256, 2, 1
    a.x, a.dt, a.A, a.B, a.C, a.out, a.states = (addr(i) for i in range(20, 27))
    a.io_dtype, a.dt_dtype, a.state_dtype = _abi.SSU_BF16, _abi.SSU_F32, _abi.SSU_F32
    a.dt_min, a.dt_max = 0.0, float("inf")
    a.cu_chunk_seqlens, a.seq_idx, a.last_chunk_indices = addr(30), addr(31), addr(32)
    a.meta_dtype = _abi.SSU_I32
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_ssd_noalloc_host_checks(lib):
    """The static-scratch prefill refuses a caller workspace and calls whose
    scratch exceeds SSU_SSD_STATIC_SCRATCH_BYTES before touching any device; the
    header's constant is what the library enforces."""
    text = open(os.path.join(ROOT, "include", "ssd.h")).read()
    m = re.search(r"#define SSU_SSD_STATIC_SCRATCH_BYTES \(\(size_t\)(\d+) << (\d+)\)", text)
    cap = int(m.group(1)) << int(m.group(2))
    a = _ssd_args(workspace=addr(40), workspace_bytes=1 << 20)
    assert lib.ssu_ssd_prefill_noalloc(ctypes.byref(a), None) == INV
    assert "static scratch" in lib.ssu_last_error().decode()
    # The largest chunk count that fits, and one more.
    n = 1
    while lib.ssu_ssd_workspace_bytes(n + 1, 1, 128, 64, 128, 8, 128) <= cap:
        n += 1
    a = _ssd_args(nheads=128, ngroups=8, chunk_size=128, nchunks=n + 1, tokens=128 * (n + 1))
    assert lib.ssu_ssd_prefill_noalloc(ctypes.byref(a), None) == UNS
    msg = lib.ssu_last_error().decode()
    assert "static scratch holds" in msg and str(cap) in msg, msg
    assert n == 34, n


def test_ssd_workspace_of_a_recorded_call_host(monkeypatch):
    """A prefill recorded into a graph gets scratch of its own: later calls neither replace
    nor share it, and it replaces no buffer of the calls outside."""
    import types

    import torch
    capturing = [False]
    empty = torch.empty
    monkeypatch.setattr(ssu, "_ssd_workspaces", {})
    monkeypatch.setattr(torch, "empty", lambda *s, dtype, device: empty(*s, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=5))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: __import__("contextlib").nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    device = torch.device("cuda", 0)
    outside = ssu._cached_workspace(device, 100)
    capturing[0] = True
    first, second = ssu._cached_workspace(device, 100), ssu._cached_workspace(device, 1000)
    capturing[0] = False
    assert first is not outside and first is not second and second.numel() == 1000 + 255
    assert list(ssu._ssd_workspaces.values()) == [outside]
    assert ssu._cached_workspace(device, 50) is outside
    assert ssu._cached_workspace(device, 1000) is not second


def test_calls_run_on_the_tensors_gpu_host(monkeypatch):
    """A call on tensors of a GPU that is not current makes it current for the launch (a default
    stream's handle does not name a GPU); on the current one it switches nothing."""
    import contextlib
    import types

    import torch
    current, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d.index
        yield
        current[0] = before

    monkeypatch.setattr(ssu, "_several_gpus", True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d: types.SimpleNamespace(cuda_stream=100 + d.index))

    def entry(ref, stream):
        seen.append((current[0], stream.value))
        return _abi.SSU_OK

    call = ssu.PreparedCall.__new__(ssu.PreparedCall)
    call._entry, call._fn, call._ref, call.out = "ssu_one_token", entry, None, "out"
    for index in (0, 1):
        call._device = torch.device("cuda", index)
        assert call() == "out" and call(types.SimpleNamespace(cuda_stream=7)) == "out"
    assert seen == [(0, 100), (0, 7), (1, 101), (1, 7)] and current == [0]
