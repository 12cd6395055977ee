"""The stored HBM counters belong to the convolutions' sources, and to no others."""
import os

import bench


def test_the_counters_are_of_the_current_sources():
    for call in ("fwd1", "bwd1", "dgrad1", "wgrad1"):
        assert bench.measured_traffic(bench.DEFAULT_WORKLOAD, call) > 0


def test_the_digest_covers_the_convolutions_alone():
    names = set(bench.conv_sources())
    assert {"gc_api.hip", "fwd_ws_f32.hip", "bwd_fused_bf16.hip", "wgrad_rf_f32_dev.h", "gc_kernels.h", "ig_common.h"} <= names
    assert not names & {"gc_train.h", "gc_train_api.hip", "gc_vec.h", "gc_norm.h", "gc_embed.h"}
    csrc = os.path.join(bench.ROOT, "backward_implicit_gemm_amd", "csrc")
    others = [n for n in os.listdir(csrc) if n not in names]
    assert others and all(n.startswith(("embed", "norm", "grad", "gc_")) for n in others)


def test_the_digest_changes_with_a_source(monkeypatch):
    was, sources = bench.source_digest(), bench.conv_sources()
    sources["ig_common.h"] += "\n"
    monkeypatch.setattr(bench, "conv_sources", lambda: sources)
    assert bench.source_digest() != was
    assert bench.measured_traffic(bench.DEFAULT_WORKLOAD, "fwd1") is None
