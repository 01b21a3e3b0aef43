"""Properties of the gfx950 code that the optimizer and 4-bit kernels compile to
(CPU only): no scratch, no packed fp32, wide accesses whatever the alignment,
and, in the tiled product, accumulators that stay where they are, waits only
where they are written, and matrix instructions of the 4-bit format."""
import os
import re
import subprocess
import tempfile

import pytest

from gradient_sync_amd import _build as B

SOURCES = ["optim_kernels.hip", "mxfp4_quant.hip", "mxfp4_gemm.hip"]


@pytest.fixture(scope="module")
def kernels():
    out = {}
    with tempfile.TemporaryDirectory() as tmp:
        procs = []
        for src in SOURCES:
            asm = os.path.join(tmp, src + ".s")
            cmd = [B.HIPCC, *B.FLAGS, "-I", B.CSRC, "-I", os.path.join(B.ROOT, "include"), "--cuda-device-only", "-S",
                   os.path.join(B.CSRC, src), "-o", asm]
            procs.append((asm, subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)))
        for asm, p in procs:
            assert p.wait() == 0, asm
            text = open(asm).read()
            for m in re.finditer(r"\.amdhsa_kernel (\S+)(.*?)\.end_amdhsa_kernel", text, re.S):
                start = re.search(r"^" + re.escape(m.group(1)) + r":", text, re.M).start()
                out[m.group(1)] = (m.group(2), text[start:text.index(".Lfunc_end", start)])
    return out


def pick(kernels, part):
    found = {n: v for n, v in kernels.items() if part in n}
    assert found, part
    return found


def test_no_scratch_and_no_packed_fp32(kernels):
    assert len(kernels) >= 28
    for name, (desc, body) in kernels.items():
        assert int(re.search(r"private_segment_fixed_size (\d+)", desc).group(1)) == 0, name
        assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", body), name


def test_wide_accesses(kernels):
    for name, (_, body) in pick(kernels, "grad_norm_kernel").items():
        assert re.search(r"global_load_dwordx4 .* nt", body), name
    for name, (_, body) in pick(kernels, "adamw_kernelILi0ELi0ELb0").items():
        assert len(re.findall(r"global_load_dwordx4 .* nt", body)) >= 8, name
        assert len(re.findall(r"global_store_dwordx4 .* nt", body)) >= 6, name
    for name, (_, body) in pick(kernels, "mxfp4_quantize").items():
        assert "global_load_dwordx4" in body, name


def test_the_norm_neither_writes_back_nor_drops_caches(kernels):
    for name, (_, body) in pick(kernels, "grad_norm_kernel").items():
        assert not re.search(r"\bbuffer_(wbl2|inv)\b", body), name


def test_tiled_product_loop(kernels):
    """From the first matrix instruction to the last: one pass of the loop over K, and in the kernel that
    goes through several tiles the choice of the next one."""
    for name, (_, body) in pick(kernels, "mxfp4_gemm_tile_kernel").items():
        lines = body.splitlines()
        at = [i for i, ln in enumerate(lines) if "v_mfma" in ln]
        loop = "\n".join(lines[at[0]:at[-1] + 1])
        wb, several = 8 if "tile_kernelILi8" in name else 4, "ELb1EEE" in name
        assert len(at) == 4 * wb * wb, name
        assert len(re.findall(r"v_mfma_scale_f32_16x16x128_f8f6f4 a\[.* cbsz:4 blgp:4", loop)) == len(at), name
        assert not re.search(r"\bv_accvgpr", loop), name
        assert len(re.findall(r"\bs_barrier\b", body)) == 5, name       # four in the loop, one before it
        if not several:
            assert len(re.findall(r"s_waitcnt vmcnt", loop)) == 4, name
            # nothing but the choice of scale bytes between the matrix instructions
            valu = {m for m in re.findall(r"^\s*(v_\w+)", loop, re.M) if not m.startswith("v_mfma")}
            assert valu == {"v_perm_b32"}, (name, valu)


def test_counted_stores(kernels):
    """The kernel that goes through several tiles counts its stores of the tile before where it waits for
    loads: 32 of them, and no other access to memory than the loads it counts."""
    for name, (_, body) in pick(kernels, "mxfp4_gemm_tile_kernelILi8ELi1ELb1ELb1E").items():
        assert len(re.findall(r"\bglobal_store_dwordx4\b", body)) == 32, name
        assert not re.search(r"\b(global_load|flat_|scratch_|global_atomic)", body), name
        assert len(re.findall(r"\bglobal_store", body)) == 32, name


def test_few_row_products_branch_by_scalars(kernels):
    """A matrix instruction runs whatever the lane mask says: what skips one is a jump, not a mask."""
    for name, (_, body) in pick(kernels, "mxfp4_gemm_few_kernel").items():
        lines = body.splitlines()
        for i, ln in enumerate(lines):
            if "v_mfma" not in ln:
                continue
            for back in reversed(lines[:i]):
                if re.match(r"\.LBB", back) or "v_mfma" in back or "s_cbranch" in back:
                    break
                assert "saveexec" not in back, name


def test_tiles_in_turn_loop(kernels):
    """The kernels that go through several tiles, pass by pass: between the matrix instructions of their loop over
    K stands nothing but the choice of scale bytes; the choice of the next tile is one block apart, which a
    pass that is not a tile's last jumps over; scalars kept in vector lanes are fetched outside the loop."""
    several = {n: v for n, v in pick(kernels, "mxfp4_gemm_tile_kernelILi8").items() if "ELb1EEE" in n}
    assert len(several) == 3
    for name, (_, body) in several.items():
        blocks = re.split(r"^(?=\.LBB\S+:|; %bb\.)", body, flags=re.M)
        loop = [b for b in blocks if "Depth=2" in "\n".join(b.splitlines()[:3])]
        assert sum(b.count("v_mfma") for b in loop) == body.count("v_mfma") == 256, name
        vector = lambda b: set(re.findall(r"^\s*(v_\w+)", b, re.M)) - {"v_mfma_scale_f32_16x16x128_f8f6f4"}
        change = []
        for b in loop:
            if "v_mfma" in b:
                assert vector(b) <= {"v_perm_b32"}, (name, vector(b))
            elif vector(b):
                change.append(b)
        assert len(change) == 1 and vector(change[0]) == {"v_mov_b32_e32"}, (name, [vector(b) for b in change])
        assert len(re.findall(r"\bv_mov_b32", change[0])) <= 32, name
        before = loop[loop.index(change[0]) - 1]
        assert re.search(r"\bs_cbranch", before) and "v_mfma" not in before, name
        # where the tile before left stores on their way, they are counted on top: in the two waits of an even stage
        waits = sorted(int(n) for b in loop for n in re.findall(r"s_waitcnt vmcnt\((\d+)\)", b))
        if "ILi8ELi1ELb1" in name:
            assert len(waits) == 6 and waits[4] - 32 in waits[:4] and waits[5] - 32 in waits[:4], (name, waits)
        else:
            assert len(waits) == 4, (name, waits)
