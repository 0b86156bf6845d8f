"""The benchmark reports the traffic reading that is committed: it was taken on the
GEMM sources as they are."""
import importlib.util
import json
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_committed_reading_is_of_these_sources():
    spec = importlib.util.spec_from_file_location("bench", os.path.join(ROOT, "bench.py"))
    bench = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bench)
    with open(os.path.join(ROOT, "profiles", "traffic_sparse_gemm_mlp_up.json")) as f:
        assert bench.load_traffic("mlp_up") == json.load(f)
