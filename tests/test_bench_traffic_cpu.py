"""bench.py's traffic figure stands only while every source of the kernel that it
was counted on is unchanged (CPU only)."""

from __future__ import annotations

import json
import os
import re

import pytest

import bench

GEMM = "gram_memory_layer_engram_amd/csrc/gemm.hip"
KERNEL = "gemm_bf16_kernel_gate_epilogue"


def _included(rel):
    """The file and what it includes from its own folder, one level down each."""
    todo, seen = [rel], []
    while todo:
        f = todo.pop()
        if f in seen:
            continue
        seen.append(f)
        text = open(os.path.join(bench.ROOT, f)).read()
        todo += [os.path.join(os.path.dirname(f), m) for m in re.findall(r'#include "([^"/]+)"', text)]
    return seen


@pytest.fixture
def tree(tmp_path, monkeypatch):
    files = _included(GEMM)
    for f in files:
        os.makedirs(tmp_path / os.path.dirname(f), exist_ok=True)
        (tmp_path / f).write_bytes(open(os.path.join(bench.ROOT, f), "rb").read())
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    monkeypatch.setattr(bench, "TRAFFIC_FILE", str(tmp_path / "traffic.json"))
    (tmp_path / "traffic.json").write_text(json.dumps(
        {KERNEL: {"source_sha": bench._source_sha(bench.GEMM_SOURCES), "hbm_bytes_per_launch": 5}}))
    return tmp_path


def test_every_gemm_source_counts(tree):
    assert bench._traffic(KERNEL, bench.GEMM_SOURCES) == 5
    # common.h: shared declarations of every kernel, none of the GEMM's stores or loads
    for f in set(_included(GEMM)) - {"gram_memory_layer_engram_amd/csrc/common.h"}:
        before = (tree / f).read_bytes()
        (tree / f).write_bytes(before + b"\n")
        assert bench._traffic(KERNEL, bench.GEMM_SOURCES) is None, f
        (tree / f).write_bytes(before)
    assert bench._traffic(KERNEL, bench.GEMM_SOURCES) == 5


def test_records_name_the_sources():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        rec = json.load(f)
    for k in ("gemm_bf16_kernel", KERNEL):
        assert rec[k]["sources"] == list(bench.GEMM_SOURCES)
