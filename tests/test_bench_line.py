"""bench.py's line on standard output is the headline alone, and short (CPU)."""
import importlib.util
import json
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bench():
    spec = importlib.util.spec_from_file_location("bench_line", os.path.join(ROOT, "bench.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_headline_is_one_short_line(capsys, monkeypatch):
    bench = _bench()
    # the longest of each kind: a sentence, numbers in full
    text, number = "x" * 300, 12345678.123456789
    block = {f"key_{i}": number for i in range(10)}
    keys = ("metric unit data dtype scaling higher_is_better vs_baseline n_gpus steps warmup ms_per_step "
            "ms_per_step_median ms_per_step_min value steps_per_s resampled_prompts_per_step mean_ess "
            "mean_ess_over_n gpu_launches").split()
    out = {k: number for k in keys} | {"step_timing": text, "config": block, "roofline": block, "step_roofline": block,
                                       "clocks": block, "e2e": block, "extensions": {f"e{i}": block for i in range(8)},
                                       "workloads": {f"w{i}": block for i in range(80)}}
    monkeypatch.setattr(bench, "parse_args", lambda: type("A", (), dict(
        impl="ours", gpus=1, no_cpu_baseline=False, cpu_seconds=1.0))())
    monkeypatch.setattr(bench, "dist_setup", lambda gpus: (1, 0, 0))
    monkeypatch.setattr(bench, "run_ours", lambda *a: dict(out))
    monkeypatch.setattr(bench, "workload", lambda args: None)
    monkeypatch.setattr(bench, "cpu_baseline", lambda *a: {**block, "sample": text, "parity_sample": block})
    assert bench.main() == 0
    got = capsys.readouterr()
    lines = got.out.splitlines()
    assert len(lines) == 1 and len(lines[0]) < 4096
    headline = json.loads(lines[0])
    assert set(out) - set(bench.DETAILS) | {"cpu_baseline", "parity_sample"} == set(headline)
    assert json.loads(got.err) == {k: out[k] for k in bench.DETAILS}
