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
