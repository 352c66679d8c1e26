"""Tensor-memory allocations wait without a limit, so no two CTAs whose columns together exceed
an SM's 512 may share one (csrc/sm100_ptx.cuh, tmem_alone). Nothing here runs on a GPU: every
kernel that allocates is held to the rule where it is compiled."""

import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "diffusion_transformer_moe_b200" / "csrc"
SOURCES = sorted(p.name for p in CSRC.glob("*.cu") if "tmem_alloc" in p.read_text())


def test_the_allocating_kernels_are_these():
    assert SOURCES == ["experts_sm100.cu", "linear.cu", "router_sm100.cu"]


@pytest.mark.parametrize("name", SOURCES)
def test_kernels_that_take_all_columns_leave_no_room_for_another(name):
    text = (CSRC / name).read_text()
    # one allocation of all 512 columns, one check of its kernel's shared memory
    wide = [a for a in re.findall(r"tmem_alloc(?:_pair)?\(&tmem_base_sh, ([^)]+)\)", text)
            if a != "tmem_cols"]
    assert len(wide) == len(re.findall(r"static_assert\(tmem_alone\(", text)) > 0


def test_the_narrow_tiles_ask_for_the_least_that_keeps_others_away():
    ptx = (CSRC / "sm100_ptx.cuh").read_text()
    sm, least = (int(re.search(rf"constexpr size_t {n} = (\d+);", ptx).group(1))
                 for n in ("kSmSmem", "kTmemLeastSmem"))
    assert sm == 228 * 1024 and 2 * (least + 1024) < sm < 3 * (least + 1024)
    # the router's smallest ring: six stages of 128 x 64 tokens and 64 x 64 weights in bf16
    assert 6 * (128 + 64) * 64 * 2 + 1024 + least + 1024 > sm
    linear = (CSRC / "linear.cu").read_text()
    assert "if (need < kTmemLeastSmem) need = kTmemLeastSmem;" in linear
    assert re.search(r"tmem_cols = p\.bn < 32 \? 32u : \(uint32_t\)p\.bn;", linear)
    for bn in re.findall(r"consider\((?:true|false), ([^;]+)\);", linear):
        assert all(int(v) <= 128 for v in re.findall(r"\b\d+\b", bn))
