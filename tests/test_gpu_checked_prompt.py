"""The prompt operators on the checked build, whose device bounds assertions
report DFLASH_ERR_CHECK in the status word: every result still matches and
every status stays as it is on the normal build."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SUITES = {
    "test_gpu_prompt_attn.py": "ragged or context or rows_of_no_sequence or few_rows or items_that_many or bad_ or "
                               "unmapped or many_short or share_a_workspace or values_that_later",
    "test_gpu_qk_norm.py": "",
    "test_gpu_logprobs.py": "",
    "test_gpu_prompt_engine.py": "",
}


@pytest.mark.parametrize("name", list(SUITES))
def test_on_the_checked_build(name):
    env = dict(os.environ, DFLASH_LIB="checked")
    code = ("import sys\n"
            f"sys.path.insert(0, {ROOT!r})\n"
            "from block_diffusion_speculative_step_gb300 import dflash as D\n"
            "assert D.dflash_build_flags() == D.DFLASH_BUILD_CHECKED, 'not the checked library'\n"
            "import pytest\n"
            f"sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', '-m', 'gpu', {os.path.join(ROOT, 'tests', name)!r}, "
            f"'-k', {SUITES[name]!r}]))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
