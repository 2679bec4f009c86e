"""The KV cache writer's division-free K codes, checked on the host: every bf16
value up to the row's maximum, for every mantissa of the maximum at exponents
across the range (``k_quotient_check all`` covers every maximum)."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_corrected_quotient_codes_equal_the_division(tmp_path):
    exe = str(tmp_path / "k_quotient_check")
    subprocess.run(["gcc", "-O2", "-ffp-contract=off", "-fno-fast-math", "-fopenmp", "-std=c11",
                    os.path.join(HERE, "k_quotient_check.c"), "-o", exe, "-lm"], check=True)
    out = subprocess.run([exe, "sample"], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stdout[-2000:]
    assert int(out.stdout.split("pairs ")[1].split()[0]) > 30_000_000, out.stdout
    assert "differ 0" in out.stdout, out.stdout
