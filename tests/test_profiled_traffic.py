"""The DRAM traffic that the bench lines quote comes from captures of the kernels as they are."""
import json
import os

import pytest

import bench


def entries(name):
    with open(os.path.join(bench.PROFILES, name)) as f:
        return sorted(json.load(f))


@pytest.mark.parametrize("workload", entries("decode_traffic.json"))
def test_decode_captures_belong_to_the_sources(workload):
    assert bench.profiled_traffic(workload) is not None


@pytest.mark.parametrize("workload", entries("prefill_traffic.json"))
def test_prefill_captures_belong_to_the_sources(workload):
    assert bench.profiled_prefill_traffic(workload) is not None


def test_the_hash_covers_every_header_of_the_kernel():
    """What a kernel's file includes from its own folder, and what that includes, is hashed with it (but for launch.h,
    whose kernels' arguments and launches move no bytes)."""
    csrc = os.path.join(bench.ROOT, "paged_kv_cache_377_b200", "csrc")

    def closure(name, seen):
        with open(os.path.join(csrc, name)) as f:
            for line in f:
                if line.startswith('#include "') and os.path.exists(os.path.join(csrc, line.split('"')[1])):
                    inc = line.split('"')[1]
                    if inc not in seen and inc != "launch.h":
                        seen.add(inc)
                        closure(inc, seen)
        return seen

    import inspect
    hashed = inspect.getsource(bench.prefill_sources_sha)
    for name in closure("prefill_tc.cu", set()):
        assert f'"{name}"' in hashed, name


def test_comments_and_layout_are_not_code(tmp_path):
    a, b, c = (tmp_path / x for x in "abc")
    a.write_text("int f() { return 1; }  // one\n")
    b.write_text("/* what\n it does */\nint f() {\n    return 1;\n}\n")
    c.write_text("int f() { return 2; }  // one\n")
    assert bench.code_sha([a]) == bench.code_sha([b]) != bench.code_sha([c])
    assert bench.code_sha([a, c]) != bench.code_sha([c, a])
