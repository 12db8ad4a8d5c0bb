"""The kernels of CTA pairs: what one CTA writes and the other's products read is ordered by barriers, so every
arrival at another CTA's barrier has to release to the cluster, and the waits on barriers of the pair to
acquire from it.  (Without a scope both are the CTA's own.  No run shows the difference; the sources do.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kda_decode_recurrence_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_arrivals_at_another_ctas_barrier_release_to_the_cluster():
    found = 0
    for name in sorted(os.listdir(CSRC)):
        text = source(name)
        for at in [m.start() for m in re.finditer(r"mbarrier\.arrive[.\w:]*", text)]:
            op = re.match(r"mbarrier\.arrive[.\w:]*", text[at:]).group()
            if "shared::cluster" not in op:
                continue
            found += 1
            before = text[:at][text[:at].rfind("asm"):]
            assert ".release.cluster" in op or (".relaxed.cluster" in op and "fence.release.sync_restrict::shared::cta.cluster" in before), \
                f"{name}: {op}"
    assert found > 0


def test_waits_of_the_pair_kernels_acquire_from_the_cluster():
    for name in ("kda_attn_latent.cu", "kda_attn_expanded.cu", "kda_attn_tree_pairs.cu"):
        text = source(name)
        assert "wait_together<true>(" in text and not re.search(r"wait_together\(", text), name
        # plain waits: for notes (the CTA's own warps), and for copies and products in flight before the CTA leaves
        for bar in re.findall(r"mbar_wait\((&?[\w.]+)", text):
            assert bar.split(".")[-1] in ("part_empty", "value_full", "key_full", "key_ready", "q_ready", "done"), f"{name}: {bar}"
    assert "acquire.cluster" in source("kda_async.cuh")
