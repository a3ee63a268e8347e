"""Shared memory that threads use by ordinary accesses and that bulk or tensor copies
write afterwards: a barrier alone does not order the two, so every thread fences the
proxies between its last access and the barrier in front of the copies."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_moe_dispatch_layout_gb300", "csrc")
FENCE = "fence_proxy_async_smem();"


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_group_tables_built_where_copies_land():
    """The row offsets' scan borrows memory of the stages in the kernels that copy by
    tensor maps.  (In memory of its own it needs no fence; nor in linear_i8.cu's first
    stages, which threads alone write, fenced before the products read them.)"""
    borrowed = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = _code(os.path.basename(path))
        for call in re.finditer(r"build_group_tables<\w+>\(([^;]*)\);", text):
            scan = call.group(1).split(",")[-4].strip()
            if scan == "s_scan":
                assert re.search(r"__shared__ \w+ s_scan\[", text), path
                continue
            assert scan == "smem", path
            if path.endswith("linear_i8.cu"):
                assert text.count("sbase + St::kOffBytes + s * St::kByteBytes") == 2
                assert "kOffBytes = kF16 * kF16Bytes" in text
                continue
            borrowed += 1
            assert FENCE in text[call.end():text.index("__syncthreads();", call.end())], path
    assert borrowed == 1
    text = _code("gmm.cu")
    assert "s_r = reinterpret_cast<int64_t*>(smem + kOffA)" in text
    last = text.rindex("s_t[tid]")
    assert FENCE in text[last:text.index("__syncthreads();", last)]


def test_rows_staged_for_a_copy_out():
    """What threads stage for a tensor copy to memory."""
    for unit in ("linear_f8.cu", "gmm.cu"):
        text = _code(unit)
        for store in re.finditer(r"tensor_store_2d\(&|tma_store_2d\(&", text):
            before = text[:store.start()]
            assert before.rfind(FENCE) > before.rfind("bulk_wait_read"), unit
