"""What the sources of the serving-step kernels keep to, without a GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_hp_gb300", "csrc")
STEP = ["hp_rope.cu", "hp_step.cu", "hp_latent.cu", "hp_latent_tc.cu", "hp_latent_prefill_tc.cu", "hp_latent.cuh",
        "hp_latent_plan.cuh", "hp_scan.cuh", "hp_step.cuh"]


def code(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_read_only_loads_behind_a_kernel_that_may_still_write():
    """The first kernel of these calls is resident while the stream's last kernel still writes what it
    will read: the read-only path, which is for memory that does not change over a kernel's life, is
    not for them."""
    for name in STEP:
        text = code(name)
        assert not re.search(r"__ldg|\.nc\.|__ldcg_nc|__restrict__", text), name


def test_dependent_kernels_wait_before_they_look_at_memory():
    """Every kernel of these files waits for the one before it, on every path: the wait comes before the
    kernel's first return, read of an argument's buffer or store (what stands before it: shared memory,
    TMEM, maps, thread numbers)."""
    seen = 0
    for name in STEP:
        for m in re.finditer(r"__global__ void.*?\n\{\n(.*?)\n\}\n", code(name), re.S):
            body = m.group(1)
            at = body.find("pdl_wait();")
            assert at >= 0, (name, m.group(0)[:120])
            before = body[:at]
            assert "return" not in before and not re.search(r"a\.(hdr|units|lens|table|ws|slot_map|d_status|blocks)\b(?!;)\s*(\[|->)", before), \
                (name, before)
            seen += 1
    assert seen >= 11
