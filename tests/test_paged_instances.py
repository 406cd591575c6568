"""Which instance of a paged kernel a call runs, and what its warps do there (static checks, no GPU): what costs time without
changing a result."""
import os
import re

from tests.test_kernel_source import CSRC, block_from, code


def kernel(text, name):
    """The body of kernel `name`."""
    m = re.search(r"__global__[^{;]*\b%s\s*\(" % name, text)
    return block_from(text, m.start())


def test_keys_stored_as_they_come_have_instances_of_their_own():
    """Registers, spills and prefetches that only a rotation needs slow a plain copy down by 10 to 18 % where one instance does
    both: whether keys are turned is decided at the launch, not in the kernel."""
    text = code(os.path.join(CSRC, "k_paged_append.cu"))
    assert not re.search(r"a\.rope\s*[!=]=", kernel(text, "k_paged_append"))
    launch = block_from(text, text.index("cudaError_t launch("))
    assert re.search(r"if \(a\.rope == nullptr\) return .*k_paged_append<T, D, true, false, kSlots>", launch)


def test_joins_work_out_waves_only_where_there_may_be_some():
    """The sums over whole items taken in waves make a join 1 us longer: calls that take none run an instance without them."""
    text = code(os.path.join(CSRC, "k_paged_join.cu"))
    assert "kvc_pg_sched<R, KVC_PG_TC_TILE, kWaves> sch;" in kernel(text, "k_paged_join")
    assert re.search(r"return a\.waves \? go\(k_paged_join<T, D, true>\) : go\(k_paged_join<T, D, false>\);", text)
    assert "pg_sched_bytes(a.B, a.waves)" in text


def test_warps_of_queries_alone_leave_the_keys_loop_out():
    """With several axes a warp that has keys goes through their loop whole (its lanes exchange positions), but one that has none
    must not: it would load head 0's keys, positions and angles for every token and store nothing."""
    body = kernel(code(os.path.join(CSRC, "k_paged_append.cu")), "k_paged_append")
    keys = body[body.index("const int page ="):]
    loop = keys.index("for (int p = lo + warp / gw; p < end; p += stride)")
    guard = re.findall(r"if \(([^\n]*)\) \{", keys[:loop])[-1]
    assert guard == "kAxes ? group < a.kv_groups : have", guard
    other = kernel(code(os.path.join(CSRC, "k_paged4_append.cu")), "k_paged4_append")
    assert re.search(r"if \(group >= a\.kv_groups\) \{\s*append_queries[^}]*return;\s*\}", other)


def test_fp32_appends_at_slots_are_launched_without_axes():
    """28 bytes of launch parameters that a kernel has no use for make an fp32 step 0.1 us longer."""
    text = code(os.path.join(CSRC, "paged_append.h"))
    plain = block_from(text, text.index("struct AppendArgs"))
    assert not re.search(r"pos\b|n_axes|pair_axis", plain)
    assert "std::conditional_t<kAxes != kSlots || sizeof(T) == 2, AxesArgs, AppendArgs>" in text
    assert "ArgsOf<T, kAxes> a)" in code(os.path.join(CSRC, "k_paged_append.cu"))
