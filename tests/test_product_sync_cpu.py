"""The CTA pair's synchronisation in csrc/moe_product.cuh, read from its source:
what no run can show, because hardware may happen to order more than the
memory model does."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def source():
    text = open(os.path.join(ROOT, "sparse_expert_gemv_gb300", "csrc", "moe_product.cuh")).read()
    return re.sub(r"//[^\n]*", "", text)


def test_arrivals_on_the_other_cta_release_at_cluster_scope():
    text = re.sub(r'"\s*"', "", source())          # joined string literals
    arrivals = re.findall(r"[^;]*;[^;]*mbarrier\.arrive\.[^;]*shared::cluster[^;]*;", text)
    arrivals = [a for a in arrivals if "tcgen05.commit" not in a]
    assert arrivals
    for a in arrivals:
        own = "mbarrier.arrive.release.cta.shared::cluster" in a
        assert own or "mbarrier.arrive.relaxed.cluster.shared::cluster" in a, a
    # a relaxed arrival follows a release fence over what it announces
    fenced = re.findall(r"fence\.release\.sync_restrict::shared::cta\.cluster;[^;]*;?[^;]*MOE_ELECT[^;]*"
                        r"mbarrier\.arrive\.relaxed\.cluster", text)
    assert len(fenced) == len(re.findall(r"mbarrier\.arrive\.relaxed\.cluster", text)) == 1


def test_only_a_barrier_of_one_cta_is_waited_for_at_cta_scope():
    text = source()
    waits = re.findall(r"mbarrier\.try_wait\.parity\.([a-z_.]+)\.shared::cta", text)
    assert sorted(set(waits)) == ["acquire.cluster", "acquire.cta"]
    own = re.findall(r"prod_wait<Arrivals::kOwn>\(&(\w+)\[", text)
    assert own == ["copied"]                      # its 128 arrivals are this CTA's copying warps
    assert re.search(r"template <Arrivals A = Arrivals::kPair>\s*__device__ __forceinline__ bool prod_wait",
                     text)


def test_no_cta_leaves_with_copies_or_mmas_in_flight():
    text = source()
    end = text[text.rindex("tc::fence_before();"):]
    order = [end.index(s) for s in ("__syncthreads();", "prod_wait_end(drain, 0, p.err);",
                                    "if (warp == 0 && *dead)", "cluster_sync();", "tmem_dealloc2")]
    assert order == sorted(order)                 # in both CTAs: no rank is asked before
    assert "rank" not in end
    # the last wait goes on when the pair is dead or its waits run out early
    body = text[text.index("void prod_wait_end("):]
    body = body[:body.index("\n}")]
    assert "dead" not in body and "polls" not in body.replace("kMbarPolls", "")


def test_a_timeout_marks_both_ctas():
    text = source()
    body = text[text.index("bool prod_wait(uint64_t* bar"):]
    body = body[:body.index("\n}")]
    assert "st.relaxed.cluster.shared::cluster" in body and "(blockIdx.x & 1) ^ 1" in body


def test_null_handles_are_refused():
    import ctypes
    import __graft_entry__
    b = __graft_entry__._build_module()
    if b.stale(b.OUT):
        b.build()
    from sparse_expert_gemv_gb300._lib import lib
    assert lib.moe_product_arm_timeout(None) == 1
    flags = ctypes.c_uint32(7)
    assert lib.moe_product_get_error_latest(None, ctypes.byref(flags)) == 1 and flags.value == 0
