"""include/attention.h and include/batch.h on the host: exports, struct layout, and the refusal
of every invalid call before anything reaches the GPU (addresses are fake and never
dereferenced); the bindings' refusals; and properties of the generated gfx950 code."""
import ctypes
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import selective_state_update_ssu_amd as ssu
from selective_state_update_ssu_amd import _abi, attention, build
from test_layer_host import addr, call

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
INV, UNS, OK = _abi.SSU_ERR_INVALID_ARGUMENT, _abi.SSU_ERR_UNSUPPORTED, _abi.SSU_OK


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssu.library_path()):
        build.build()
    return ssu.library()


@pytest.mark.parametrize("header,exports", [("attention.h", _abi.ATTENTION_EXPORTS),
                                            ("batch.h", _abi.BATCH_EXPORTS)])
def test_exports_every_declared_function(lib, header, exports):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, header)).read(), flags=re.S)
    names = re.findall(r"^(?:int|size_t)\s+(ssu_\w+)\s*\(", text, re.M)
    assert sorted(names) == sorted(exports)
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layout_matches_header(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "attention.h"',
             '#include "batch.h"', "int main(void){"]
    want = {}
    for cname, cls in (("ssu_attention_args", _abi.AttentionArgs), ("ssu_verify_args", _abi.VerifyArgs),
                       ("ssu_plan_args", _abi.PlanArgs)):
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        want[cname] = ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            lines.append(f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));')
            want[f"{cname}.{f}"] = getattr(cls, f).offset
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{INCLUDE}", str(src), "-o", str(exe)],
                   check=True)
    text = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert {k: int(v) for k, v in (l.split() for l in text.splitlines())} == want


def attend(lib, entry, **kw):
    varlen, packed = entry == "varlen", entry == "packed"
    a = _abi.AttentionArgs(
        struct_size=ctypes.sizeof(_abi.AttentionArgs), state_dtype=_abi.SSU_F32, state=addr(1),
        nslots=64, slot_stride=4 * 32 * 64, rows=10, nheads=4, ngroups=2, key_dim=64, value_dim=32,
        q=addr(2), k=addr(3), v=addr(4), out=addr(5), q_stride=128, k_stride=128, v_stride=128,
        out_stride=128, io_dtype=_abi.SSU_BF16, beta_dtype=_abi.SSU_F32, decay=addr(6),
        decay_stride=4, beta=addr(7), beta_stride=4, scale=0.125,
        nseq=10 if entry == "update" else 3, cu_seqlens=None if entry == "update" else addr(8),
        has_initial=addr(9) if varlen else None, slots=addr(10), pad_slot_id=-1)
    if varlen:
        a.workspace, a.workspace_bytes = addr(13), 1 << 33
    if packed:
        a.slot_seq_stride, a.slot_step_stride, a.num_accepted = 4, 1, addr(11)
        a.dst, a.dst_seq_stride, a.dst_step_stride, a.steps = addr(12), 4, 1, 4
    return call(lib, f"ssu_attention_{entry}", a, kw)


@pytest.mark.parametrize("entry,kw,code,needle", [
    ("varlen", dict(struct_size=8), INV, "struct_size"),
    ("varlen", dict(reserved=1), INV, "reserved"),
    ("varlen", dict(io_dtype=3), INV, "io_dtype"),
    ("varlen", dict(state_dtype=-1), INV, "state_dtype"),
    ("varlen", dict(beta_dtype=_abi.SSU_F16), INV, "beta"),
    ("varlen", dict(rows=-1), INV, "sizes"),
    ("varlen", dict(nheads=0), INV, "sizes"),
    ("varlen", dict(nslots=0), INV, "sizes"),
    ("varlen", dict(nseq=-1), INV, "sizes"),
    ("varlen", dict(ngroups=3), INV, "multiple"),
    ("varlen", dict(key_dim=60), UNS, "key_dim"),
    ("varlen", dict(key_dim=264), UNS, "key_dim"),
    ("varlen", dict(value_dim=257), UNS, "value_dim"),
    ("varlen", dict(rows=1 << 31), UNS, "2^30"),
    ("varlen", dict(slot_stride=4 * 32 * 64 - 1), INV, "slot_stride"),
    ("varlen", dict(q_stride=-1), INV, "strides"),
    ("varlen", dict(out_stride=127), INV, "out_stride"),
    ("varlen", dict(cu_dtype=2), INV, "cu_dtype"),
    ("varlen", dict(slot_dtype=2), INV, "slot_dtype"),
    ("varlen", dict(cu_seqlens=None), INV, "cu_seqlens must not"),
    ("varlen", dict(q=None), INV, "q must not"),
    ("varlen", dict(decay=None), INV, "decay must not"),
    ("varlen", dict(state=None), INV, "state must not"),
    ("varlen", dict(out=None), INV, "out must not"),
    ("varlen", dict(v=addr(4) + 1), INV, "v must be aligned"),
    ("varlen", dict(out=addr(5) + 1), INV, "out must be aligned"),
    ("varlen", dict(state=addr(1) + 8), UNS, "16-byte"),
    ("varlen", dict(slot_stride=4 * 32 * 64 + 1), UNS, "16-byte"),
    ("varlen", dict(out=addr(4)), INV, "out overlaps v"),
    ("varlen", dict(state=addr(2)), INV, "state overlaps q"),
    ("varlen", dict(out=addr(1)), INV, "state overlaps out"),
    ("varlen", dict(num_accepted=addr(11)), INV, "belong to ssu_attention_packed"),
    ("varlen", dict(dst=addr(11)), INV, "belong to ssu_attention_packed"),
    ("update", dict(cu_seqlens=addr(8)), INV, "update has no cu_seqlens"),
    ("update", dict(nseq=9), INV, "nseq must equal rows"),
    ("update", dict(has_initial=addr(9)), INV, "belong to ssu_attention_varlen"),
    ("update", dict(workspace=addr(13)), INV, "belong to ssu_attention_varlen"),
    ("packed", dict(slots=None), INV, "needs a slot table"),
    ("packed", dict(steps=0), INV, "steps"),
    ("packed", dict(dst_dtype=2), INV, "dst_dtype"),
    ("packed", dict(dst_step_stride=-1), INV, "table strides"),
    ("packed", dict(state=addr(12)), INV, "state overlaps dst"),
    ("packed", dict(out=addr(10)), INV, "out overlaps slots"),
])
def test_attention_rejects(lib, entry, kw, code, needle):
    rc, msg = attend(lib, entry, **kw)
    assert rc == code, (rc, msg)
    assert needle in msg, msg


@pytest.mark.parametrize("entry", ["varlen", "update", "packed"])
def test_attention_without_work(lib, entry):
    rc, msg = attend(lib, entry, rows=0, nseq=0, q=None, k=None, v=None, out=None)
    assert rc == OK, msg
    if entry != "update":
        assert attend(lib, entry, nseq=0)[0] == OK


def test_null_arguments(lib):
    for entry in _abi.ATTENTION_EXPORTS + _abi.BATCH_EXPORTS:
        if not entry.endswith("workspace_bytes"):
            assert getattr(lib, entry)(None, None) == INV, entry


def verify(lib, **kw):
    a = _abi.VerifyArgs(
        struct_size=ctypes.sizeof(_abi.VerifyArgs), target_dtype=_abi.SSU_BF16, target=addr(1),
        target_stride=1000, rows=9, vocab=1000, nseq=3, window=4, cu_seqlens=addr(2),
        drafts=addr(3), draft_seq_stride=4, draft_step_stride=1, draft_probs=addr(4),
        probs_seq_stride=4000, probs_step_stride=1000, uniforms=addr(5), uniform_stride=5,
        temperature=addr(6), tokens=addr(7), num_accepted=addr(8), workspace=addr(9),
        workspace_bytes=1 << 20)
    return call(lib, "ssu_verify_drafts", a, kw)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(struct_size=8), INV, "struct_size"),
    (dict(reserved=1), INV, "reserved"),
    (dict(target_dtype=3), INV, "target_dtype"),
    (dict(probs_dtype=3), INV, "probs_dtype"),
    (dict(cu_dtype=2), INV, "cu_dtype"),
    (dict(draft_dtype=2), INV, "draft_dtype"),
    (dict(vocab=0), INV, "sizes"),
    (dict(rows=-1), INV, "sizes"),
    (dict(window=-1), INV, "sizes"),
    (dict(window=1 << 20), UNS, "window"),
    (dict(vocab=(1 << 31) - 1), UNS, "vocab"),
    (dict(probs_step_stride=-1), INV, "strides"),
    (dict(target=None), INV, "target must not"),
    (dict(drafts=None), INV, "drafts must not"),
    (dict(uniforms=None), INV, "uniforms must not"),
    (dict(cu_seqlens=None), INV, "cu_seqlens must not"),
    (dict(tokens=None), INV, "tokens and num_accepted"),
    (dict(target=addr(1) + 1), INV, "target must be aligned"),
    (dict(tokens=addr(7) + 2), INV, "aligned"),
    (dict(workspace=None), INV, "workspace"),
    (dict(workspace_bytes=16), INV, "workspace"),
    (dict(workspace=addr(9) + 16), INV, "workspace"),
    (dict(tokens=addr(3)), INV, "tokens overlaps drafts"),
    (dict(num_accepted=addr(7) + 8), INV, "num_accepted overlaps tokens"),
    (dict(workspace=addr(1)), INV, "workspace overlaps target"),
    (dict(rows=1 << 30, target_stride=0), INV, "workspace"),
])
def test_verify_rejects(lib, kw, code, needle):
    rc, msg = verify(lib, **kw)
    assert rc == code, (rc, msg)
    assert needle in msg, msg


def test_verify_without_work(lib):
    assert verify(lib, nseq=0)[0] == OK


def plan(lib, **kw):
    a = _abi.PlanArgs(
        struct_size=ctypes.sizeof(_abi.PlanArgs), lengths=addr(1), context=addr(2), nseq=3, rows=10,
        chunk_size=4, nchunks=5, block_table=addr(3), table_stride=6, table_width=6, block_size=2,
        cu_seqlens=addr(4), row_seq=addr(5), row_pos=addr(6), row_slots=addr(7),
        cu_chunk_seqlens=addr(8), seq_idx=addr(9), last_chunk_indices=addr(10))
    return call(lib, "ssu_batch_plan", a, kw)


@pytest.mark.parametrize("kw,needle", [
    (dict(struct_size=8), "struct_size"),
    (dict(length_dtype=2), "length_dtype"),
    (dict(context_dtype=2), "context_dtype"),
    (dict(table_dtype=2), "table_dtype"),
    (dict(nseq=-1), "nseq"),
    (dict(rows=1 << 31), "rows"),
    (dict(chunk_size=-1), "chunk_size"),
    (dict(nchunks=1 << 31), "nchunks"),
    (dict(chunk_size=0), "chunk"),
    (dict(chunk_size=0, nchunks=0), "chunk tables need"),
    (dict(block_size=0), "block_size"),
    (dict(table_stride=-1), "table_stride"),
    (dict(block_table=None), "row_slots needs"),
    (dict(lengths=None), "lengths must not"),
    (dict(lengths=addr(1) + 2), "lengths must be aligned"),
    (dict(row_slots=addr(7) + 4), "row_slots must be aligned"),
    (dict(row_seq=addr(1)), "row_seq overlaps lengths"),
    (dict(row_pos=addr(5) + 4), "row_pos overlaps row_seq"),
    (dict(cu_chunk_seqlens=addr(3) + 8), "cu_chunk_seqlens overlaps block_table"),
])
def test_plan_rejects(lib, kw, needle):
    rc, msg = plan(lib, **kw)
    assert rc == INV, (rc, msg)
    assert needle in msg, msg


# ----------------------------------------------------------------------- bindings

def test_bindings_refuse_host_tensors():
    t = torch.zeros(2, 1, 8)
    state = torch.zeros(2, 1, 8, 8)
    for f, args in ((ssu.linear_attention_update, ()), (ssu.linear_attention_varlen, (torch.zeros(3),)),
                    (ssu.linear_attention_packed, (torch.zeros(3),))):
        with pytest.raises(ValueError, match="must be on a GPU"):
            f(state, t, t, t, torch.zeros(1), *args)
    with pytest.raises(ValueError, match="must be on a GPU"):
        ssu.verify_drafts(torch.zeros(2, 5), torch.zeros(1, 1), torch.zeros(1, 2), torch.zeros(2))
    with pytest.raises(ValueError, match="must be on a GPU"):
        ssu.batch_plan(torch.zeros(3, dtype=torch.int32), 5)


def test_bindings_refuse_what_is_no_tensor():
    t = torch.zeros(2, 1, 8)
    with pytest.raises(ValueError, match="q must be a tensor"):
        ssu.linear_attention_update(torch.zeros(2, 1, 8, 8), 3, t, t, torch.zeros(1))
    with pytest.raises(ValueError, match="cu_seqlens must be"):
        ssu.linear_attention_varlen(torch.zeros(2, 1, 8, 8), t, t, t, torch.zeros(1), None)
    with pytest.raises(ValueError, match="cu_seqlens must be a tensor"):
        ssu.verify_drafts(torch.zeros(2, 5), torch.zeros(1, 1), torch.zeros(1, 2), [0, 2])
    with pytest.raises(ValueError, match="nchunks needs"):
        ssu.batch_plan(torch.zeros(3, dtype=torch.int32), 5, nchunks=3)
    with pytest.raises(ValueError, match="chunk_size must be positive"):
        ssu.batch_plan(torch.zeros(3, dtype=torch.int32), 5, chunk_size=0)
    with pytest.raises(TypeError, match="arguments"):
        attention._load().plan(None)


def test_binding_switches_to_the_tensors_gpu():
    attention._load()
    names = subprocess.run(["nm", "-D", "--undefined-only", attention.binding_path()],
                           capture_output=True, text=True, check=True).stdout
    assert "device_guard_impl_registry" in names


# -------------------------------------------------------------- the generated code

UNITS = [s for s in build.SOURCES if s.startswith(("attention_", "batch_"))]


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    out = tmp_path_factory.mktemp("serve_isa")

    def one(unit):
        path = os.path.join(str(out), unit + ".s")
        flags = [f for f in build.CXXFLAGS if f not in ("-fPIC",)]
        r = subprocess.run([build.HIPCC, *flags, "--cuda-device-only", "-S",
                            os.path.join(build.CSRC, unit), "-o", path],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return unit, open(path).read()

    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    with ThreadPoolExecutor(os.cpu_count() or 1) as ex:
        return dict(ex.map(one, UNITS))


def test_no_packed_fp32_and_no_scratch(asm):
    for unit, text in asm.items():
        assert not re.search(r"v_pk_(fma|mul|add)_f32", text), unit
        sizes = re.findall(r"\.private_segment_fixed_size:\s*(\d+)", text)
        assert all(s == "0" for s in sizes), unit


def test_chunks_run_on_the_matrix_cores(asm):
    for unit, text in asm.items():
        if unit.startswith("attention_chunk"):
            assert "v_mfma_f32_16x16x32_bf16" in text, unit
            assert "ds_read_b64_tr_b16" in text, unit
