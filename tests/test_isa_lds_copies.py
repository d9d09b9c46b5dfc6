"""Inline-asm LDS copies from a scalar base, and the scans for wait states, in the gfx950 assembly of every kernel source.

A memory instruction needs five wait states after a vector instruction that wrote a scalar register it reads, and the
compiler keeps no such distance to inline asm. So each of these copies has to read its base from registers that a scalar
instruction of its own asm block wrote, whatever the compiler puts before the block. What a source includes holds copies and MFMAs too, so the scans look at
every source's assembly, not at the words in its text. Runs on the CPU; skipped where hipcc is absent.
"""
import os
import re

import test_isa_hazards as hazards
import test_isa_scalar_bases as scalar_bases
from test_isa_hazards import _device_asm, needs_hipcc
from w4a16_grouped_gemm_amd import build

_COPY = re.compile(r"global_load_lds_\w+ v\d+, (s\[\d+:\d+\]|vcc)")


def asm_blocks(asm: str):
    """The instructions of each inline-asm block, a list a block."""
    blocks, cur = [], None
    for line in asm.splitlines():
        if "#ASMSTART" in line:
            cur = []
        elif "#ASMEND" in line:
            blocks.append(cur)
            cur = None
        elif cur is not None:
            s = line.split(";")[0].strip()
            if s:
                cur.append(s)
    return blocks


def bases_from_outside(asm: str):
    """The blocks with a copy whose scalar base no scalar instruction of the block wrote; and how many such copies there are."""
    bad, copies = [], 0
    for block in asm_blocks(asm):
        for i, inst in enumerate(block):
            m = _COPY.match(inst)
            if m:
                copies += 1
                if not any(re.match(rf"s_\w+ {re.escape(m.group(1))}(,|$)", b) for b in block[:i]):
                    bad.append(block)
    return bad, copies


def sources_asm(tmp_path):
    return {os.path.basename(s): a for s, a in _device_asm(build.sources(), tmp_path).items()}


def test_scanner_flags_a_base_from_outside():
    block = "k:\n\tv_readlane_b32 s11, v40, 3\n\t;;#ASMSTART\n\ts_mov_b32 m0, s4\n\t{}\n\tglobal_load_lds_dwordx4 v2, s[10:11]\n\t;;#ASMEND\n"
    assert len(bases_from_outside(block.format("s_nop 0"))[0]) == 1
    assert len(bases_from_outside(block.format("s_mov_b64 s[12:13], s[6:7]"))[0]) == 1
    assert len(bases_from_outside(block.format("v_readlane_b32 s[10:11], v3, 1"))[0]) == 1
    assert bases_from_outside(block.format("s_mov_b64 s[10:11], s[6:7]")) == ([], 1)
    assert bases_from_outside("k:\n\tglobal_load_lds_dwordx4 v2, s[10:11]\n") == ([], 0)  # the compiler's own


@needs_hipcc
def test_copies_read_bases_that_their_own_block_wrote(tmp_path):
    bad, copies = [], {}
    for src, asm in sources_asm(tmp_path).items():
        found, copies[src] = bases_from_outside(asm)
        bad += [(src, b) for b in found]
    assert copies["grouped_gemm.hip"] > 0 and copies["grouped_wgrad.hip"] > 0
    assert not bad, f"{len(bad)} copies, e.g. {bad[:3]}"


PRODUCTS = {"grouped_gemm.hip", "grouped_wgrad.hip"}  # their copies and MFMAs are in a header that both include


@needs_hipcc
def test_wait_states_in_every_source(tmp_path):
    """Scalar writes of M0 and vector writes of bases before copies, vector writes before MFMAs."""
    with_copies, with_scalar_bases, with_mfma, bad = set(), set(), set(), []
    for src, asm in sources_asm(tmp_path).items():
        if "global_load_lds" in asm:
            with_copies.add(src)
            bad += [(src, "M0") + h for h in hazards.m0_too_close(asm)]
        found, copies = scalar_bases.short_distances(asm)
        if copies:
            with_scalar_bases.add(src)
            bad += [(src, "base") + h for h in found]
        if "v_mfma" in asm:
            with_mfma.add(src)
            bad += [(src, "MFMA") + h for h in hazards.short_distances(asm)]
    assert PRODUCTS <= with_copies and PRODUCTS <= with_scalar_bases and PRODUCTS <= with_mfma
    assert {"moe_gemm_tiled.hip", "moe_gemm_stream.hip"} <= with_copies
    assert {"moe_gemm.hip", "moe_gemm_stream.hip", "moe_gemm_tiled.hip", "mxfp4_gemm.hip"} <= with_mfma
    assert not bad, f"{len(bad)}, e.g. {bad[:5]}"


_FUNCTION = re.compile(r"^([\w$.]+):")


def unordered_exchanges(asm: str):
    """(function, first, second): LDS reads after writes, or writes after reads, of whole 16 bytes a lane with no barrier of the wave
    or the workgroup between them in the assembly's order."""
    found, name, last = [], None, None
    for line in asm.splitlines():
        m = _FUNCTION.match(line)
        if m and not line.startswith("."):
            name, last = m.group(1), None
        s = line.strip()
        if s.startswith("; wave barrier") or s.startswith("s_barrier"):
            last = None
        elif s.startswith(("ds_write_b128", "ds_read_b128")):
            kind = s.split()[0]
            if last is not None and last != kind:
                found.append((name, last, kind))
            last = kind
    return found


def test_scanner_flags_an_unordered_exchange():
    write, read, barrier = "\tds_write_b128 v1, v[2:5]\n", "\tds_read_b128 v[2:5], v1\n", "\t; wave barrier\n"
    assert len(unordered_exchanges("k:\n" + write + read)) == 1
    assert len(unordered_exchanges("k:\n" + write + barrier + read + write)) == 1
    assert unordered_exchanges("k:\n" + write + write + barrier + read + read + barrier + write) == []
    assert unordered_exchanges("k:\n" + write + "\ts_barrier\n" + read) == []


@needs_hipcc
def test_lanes_that_exchange_values_meet(tmp_path):
    """The sums of a tile leave through LDS of the wave's own: written by some lanes, read by others, overwritten by the next."""
    for src, asm in sources_asm(tmp_path).items():
        if src in PRODUCTS:
            assert "ds_write_b128" in asm and "ds_read_b128" in asm
            found = unordered_exchanges(asm)
            assert not found, (src, len(found), found[0])
