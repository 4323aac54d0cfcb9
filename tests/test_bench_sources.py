"""The traffic records of profiles/traffic.json stand for the kernels bench.py launches: an edit of another
kernel's source leaves them valid, an edit of theirs does not."""
import json
import os
import shutil

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rank_adapter_gb300", "csrc")


def test_hash_covers_the_benchmarked_kernels_only(tmp_path):
    d = str(tmp_path / "csrc")
    shutil.copytree(CSRC, d)
    before = bench.kernel_source_hash(d)
    assert before == bench.kernel_source_hash()
    for f in sorted(os.listdir(d)):
        path = os.path.join(d, f)
        text = open(path).read()
        open(path, "w").write(text + "// edited\n")
        assert (bench.kernel_source_hash(d) == before) == (f in bench.UNBENCHED_SOURCES), f
        open(path, "w").write(text)


def test_unbenched_sources_exist_and_no_other_source_includes_them():
    """Headers among them are used by one another only, but for the ABI's host code."""
    names = os.listdir(CSRC)
    assert set(bench.UNBENCHED_SOURCES) <= set(names)
    for f in set(names) - set(bench.UNBENCHED_SOURCES) - {"lora_abi.cu"}:
        text = open(os.path.join(CSRC, f)).read()
        assert not any(f'#include "{u}"' in text for u in bench.UNBENCHED_SOURCES), f


def test_records_share_one_hash():
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        rec = json.load(f)
    hashes = {k["source_hash"] for w in rec.values() for k in w.values() if isinstance(k, dict)}
    assert len(hashes) == 1
