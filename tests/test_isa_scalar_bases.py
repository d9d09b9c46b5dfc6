"""Wait states between vector instructions that write scalar registers and inline-asm copies that read them.

A memory instruction that reads a scalar register needs five wait states (issued instructions, or s_nop cycles)
after a VALU instruction that wrote it: a v_readfirstlane, or a v_readlane that brings back a register which the
compiler had set aside in a vector register. The compiler keeps that distance for its own instructions, but the LDS
copies from a scalar base are inline asm. The test compiles the sources that hold such copies to gfx950 assembly
with the library's flags and looks at what comes before each copy, along straight-line code and the branches into its
block. Runs on the CPU; skipped where hipcc is absent.
"""
import os
import re
from collections import defaultdict

from test_isa_hazards import _device_asm, _functions, _lds_dma_sources, _wait_states, needs_hipcc

NEED = 5
_COPY = re.compile(r"global_load_lds_\w+ v\d+, s\[(\d+):(\d+)\]")
_SGPR = re.compile(r"^s(?:\[(\d+):(\d+)\]|(\d+))$")


def _scalars_written(inst: str) -> set:
    """Scalar registers a VALU instruction writes: its first operand, and the carry that some have behind it."""
    op, _, rest = inst.partition(" ")
    if not op.startswith("v_"):
        return set()
    operands = [o.strip() for o in rest.split(",")]
    carry = "_co_" in op or op.startswith(("v_mad_u64", "v_mad_i64", "v_div_scale"))
    out = set()
    for o in operands[: 2 if carry else 1]:
        m = _SGPR.match(o)
        if m:
            low, high = (m.group(1), m.group(2)) if m.group(1) else (m.group(3), m.group(3))
            out.update(range(int(low), int(high) + 1))
    return out


def short_distances(asm: str):
    """(function, wait states, writer, copy) for each copy whose scalar base was written too close before it; and how
    many copies there are."""
    found, copies = [], 0
    for name, body in _functions(asm):
        insts, label_at, into = [], {}, defaultdict(list)
        for kind, v in body:
            if kind == "label":
                label_at[len(insts)] = v
            else:
                insts.append(v)
                if v.split()[0].startswith(("s_cbranch", "s_branch")):
                    into[v.split()[-1]].append(len(insts) - 1)

        def back(j, dist, base):
            hits = []
            while j >= 0 and dist < NEED:
                if base & _scalars_written(insts[j]):
                    return hits + [(dist, insts[j])]
                dist += _wait_states(insts[j])
                if j in label_at:
                    for b in into.get(label_at[j], []):
                        hits += back(b - 1, dist + 1, base)
                    if j > 0 and insts[j - 1].split()[0] == "s_branch":
                        return hits
                j -= 1
            return hits

        for i, inst in enumerate(insts):
            m = _COPY.match(inst)
            if not m:
                continue
            copies += 1
            hits = back(i - 1, 0, set(range(int(m.group(1)), int(m.group(2)) + 1)))
            found += [(name, d, w, inst) for d, w in hits]
    return found, copies


def test_scanner_flags_a_short_distance():
    copy, end = "\ts_mov_b32 m0, s4\n\ts_nop 0\n\tglobal_load_lds_dwordx4 v2, s[10:11]\n", ".Lfunc_end0:\n"
    write = "\tv_readlane_b32 s11, v40, 3\n"
    assert len(short_distances("k:\n" + write + copy + end)[0]) == 1
    assert len(short_distances("k:\n" + write + "\ts_nop 1\n" + copy + end)[0]) == 1
    assert short_distances("k:\n" + write + "\ts_nop 2\n" + copy + end) == ([], 1)
    assert short_distances("k:\n\tv_readlane_b32 s12, v40, 3\n" + copy + end) == ([], 1)
    assert len(short_distances("k:\n\tv_mad_u64_u32 v[4:5], s[10:11], v1, v2, v[4:5]\n" + copy + end)[0]) == 1
    assert len(short_distances("k:\n\tv_cmp_lt_u32_e64 s[10:11], v1, v2\n" + copy + end)[0]) == 1
    assert short_distances("k:\n\ts_add_u32 s10, s10, s3\n" + copy + end) == ([], 1)
    branchy = ("k:\n" + write + "\ts_cbranch_scc1 .LBB0_2\n\ts_nop 7\n\ts_branch .LBB0_2\n.LBB0_2:\n" + copy + end)
    assert len(short_distances(branchy)[0]) == 1


@needs_hipcc
def test_scalar_bases_are_written_early_enough(tmp_path):
    bad, copies = [], 0
    for src, asm in _device_asm(_lds_dma_sources(), tmp_path).items():
        found, n = short_distances(asm)
        copies += n
        bad += [(os.path.basename(src),) + f for f in found]
    assert copies > 0
    assert not bad, "\n".join(f"{s} {n[:60]}: {d} wait state(s): {w} -> {c}" for s, n, d, w, c in bad[:10])
